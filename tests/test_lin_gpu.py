"""Linear attention with one decay per head (kda_lin_chunk_fwd,
kda_lin_decode_step, kda_lin_bwd) on the GPU against the fp64 oracle.

Tolerances, as ||err||_2 / ||ref||_2:
  fp32 results of fp32 inputs: 1e-5, i.e. 168 half steps of 2^-24; the longest
    sums here have some 128 channels times the tokens in memory, whose
    independent roundings add up as the root of their number.
  fp32 states of bf16 inputs: 2e-5.  k v^T of bf16 values is exact in fp32;
    a kernel that splits a decayed value into two bf16 parts leaves at most
    2^-8 2^-8 = 2^-16 = 1.5e-5 of it.
  bf16 results: 4e-3.  One rounding is off by at most 2^-8 of the value, in
    the root mean square by at most 2^-8 / sqrt(3) = 2.3e-3; a result goes
    through three independent ones (the products inside a chunk, the state as
    an operand, the output): sqrt(3) 2.3e-3 = 3.9e-3.
dg of a decay per head is a sum over the tokens, whose terms have either sign
and may cancel to any smaller value.  A token's term is itself a sum over the
pairs of an earlier and a later token around it, of which neighbours share most,
so their roundings are shared too: a chunk of 128 tokens may be off by its
terms' tolerance of the sum of their magnitudes, chunks independently, however
small the whole sum is.
"""
import numpy as np
import pytest
import torch

from kda_linear_attention_fwd_b200 import kda
from oracle import linear as O
from parity import np32

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {torch.bfloat16: 4e-3, torch.float32: 1e-5}


def make(lengths, H, Hk, dk, dv, dtype, per_head=False, s0=True, seed=0):
    gen = torch.Generator().manual_seed(seed)
    T, N, dt = sum(lengths), len(lengths), DT[dtype]
    randn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    bias = -6.0 * torch.arange(H) / max(H - 1, 1)   # memories of about one to 400 tokens
    g = -torch.nn.functional.softplus(bias if per_head else bias + randn(T, H))
    cu = [0]
    for L in lengths:
        cu.append(cu[-1] + L)
    d = dict(q=unit(randn(T, Hk, dk)).to(dt), k=unit(randn(T, Hk, dk)).to(dt), v=randn(T, H, dv).to(dt), g=g.to(dt),
             s0=0.1 * randn(N, H, dk, dv) if s0 else None, dy=randn(T, H, dv).to(dt), dsf=randn(N, H, dk, dv))
    d = {k: None if x is None else x.cuda() for k, x in d.items()}
    d["cu"], d["host"] = torch.tensor(cu, dtype=torch.int32, device="cuda"), cu
    return d


def near(got, want, tol, what, room=0.0):
    a, e = np32(got).astype(np.float64), np.asarray(want, np.float64)
    assert a.shape == e.shape, (what, a.shape, e.shape)
    assert np.isfinite(a).all(), f"{what}: not finite"
    off = max(np.linalg.norm(a - e) - room, 0.0) / max(np.linalg.norm(e), 1e-30) if e.size else 0.0
    assert off <= tol, f"{what}: relative error {off:.2e} > {tol:.1e}"


def fwd_both(d, scale=0.5, **kw):
    out, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], scale=scale, initial_state=d["s0"],
                                 cu_seqlens_host=d["host"], **kw)
    ref = O.forward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], scale=scale,
                    initial_state=np32(d["s0"]))
    return out, fin, ref


SHAPES = [("bf16", 128, 128), ("bf16", 64, 128), ("bf16", 128, 64), ("bf16", 64, 64), ("f32", 128, 128),
          ("f32", 64, 128), ("f32", 128, 64), ("f32", 64, 64)]
LENGTHS = [(1,), (0, 5, 64, 0, 130), (127, 128, 129), (700, 1, 63, 65), (1111,), (0,)]


@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_prefill_matches_oracle(cuda_lib, dtype, dk, dv, lengths):
    seed = len(lengths) + sum(lengths)
    d = make(lengths, 4, 2, dk, dv, dtype, per_head=seed % 2 == 0, s0=sum(lengths) != 1111, seed=seed)
    out, fin, (o, S) = fwd_both(d)
    near(out, o, TOL[d["q"].dtype], "out")
    near(fin, S, 2e-5 if dtype == "bf16" else 1e-5, "final state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Hk", [(1, 1), (6, 2), (5, 5), (8, 1)])
def test_prefill_head_layouts(cuda_lib, dtype, H, Hk):
    d = make((200, 77), H, Hk, 64, 64, dtype, seed=H)
    out, fin, (o, S) = fwd_both(d, scale=1.0)
    near(out, o, TOL[d["q"].dtype], "out")
    near(fin, S, 2e-5 if dtype == "bf16" else 1e-5, "final state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_many_short_sequences(cuda_lib, dtype):
    """Windows that hold dozens of sequences, empty ones among them."""
    rng = np.random.default_rng(5)
    d = make(tuple(int(x) for x in rng.integers(0, 9, 150)), 3, 3, 64, 128, dtype, seed=6)
    out, fin, (o, S) = fwd_both(d)
    near(out, o, TOL[d["q"].dtype], "out")
    near(fin, S, 2e-5 if dtype == "bf16" else 1e-5, "final state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_state_in_place(cuda_lib, dtype):
    """final_state = initial_state, for sequences that cross several windows."""
    d = make((900, 3, 0, 640), 2, 2, 128, 128, dtype, seed=7)
    want, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["s0"])
    for _ in range(3):
        s = d["s0"].clone()
        out, got = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=s, final_state=s)
        assert got is s and torch.equal(out, want) and torch.equal(s, fin)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays_of_every_size(cuda_lib, dtype):
    """No decay at all, resets by -inf and by large finite values, and mixtures."""
    d = make((300, 40), 4, 4, 128, 64, dtype, seed=8)
    g = d["g"].float()
    g[:, 0] = 0.0
    g[::7, 1] = -float("inf")
    g[5::11, 2] = -500.0
    g[:, 3] *= 30.0
    g[0, 1] = -float("inf")
    d["g"] = g.to(d["g"].dtype)
    out, fin, (o, S) = fwd_both(d)
    near(out, o, TOL[d["q"].dtype], "out")
    near(fin, S, 2e-5 if dtype == "bf16" else 1e-5, "final state")
    got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], initial_state=d["s0"])
    ref = O.backward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], np32(d["dy"]),
                     initial_state=np32(d["s0"]))
    check_grads(got, ref, dtype)


def test_long_context_memory(cuda_lib):
    """A head that forgets almost nothing over 6000 tokens."""
    d = make((6000,), 2, 1, 64, 64, "f32", s0=True, seed=9)
    d["g"] = torch.full_like(d["g"], -1e-4)
    out, fin, (o, S) = fwd_both(d)
    near(out, o, 1e-5, "out")
    near(fin, S, 1e-5, "final state")


def test_continuing_from_a_state(cuda_lib):
    """Two calls over the halves of a sequence give the whole sequence's result."""
    d = make((500,), 4, 2, 128, 128, "f32", seed=10)
    whole, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["s0"])
    s, parts = d["s0"], []
    for a, b in ((0, 211), (211, 500)):
        cu = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        o, s = kda.lin_chunk_fwd(*(d[x][a:b].contiguous() for x in ("q", "k", "v", "g")), cu, initial_state=s)
        parts.append(o)
    near(torch.cat(parts), np32(whole), 1e-5, "out")
    near(s, np32(fin), 1e-5, "final state")


def test_rows_behind_the_last_sequence_are_left(cuda_lib):
    d = make((100, 60), 2, 2, 64, 64, "bf16", seed=11)
    cu = torch.tensor([0, 90, 120], dtype=torch.int32, device="cuda")
    out = torch.full_like(d["v"], 7.0)
    d["v"][120:] = float("nan")
    d["k"][120:] = float("nan")
    kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], cu, out=out)
    assert (out[120:] == 7.0).all() and torch.isfinite(out[:120]).all()


@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
@pytest.mark.parametrize("N,H,Hk,per_head", [(1, 2, 1, True), (3, 5, 5, False), (160, 4, 2, False)])
def test_decode_matches_oracle(cuda_lib, dtype, dk, dv, N, H, Hk, per_head):
    d = make((1,) * N, H, Hk, dk, dv, dtype, per_head=per_head, seed=N)
    s = d["s0"].clone()
    ref, S = O.forward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], scale=0.5,
                       initial_state=np32(d["s0"]))
    out = kda.lin_decode_step(d["q"], d["k"], d["v"], d["g"], s, scale=0.5)
    near(out, ref, TOL[d["q"].dtype], "out")
    near(s, S, 1e-6, "state")


def test_decode_steps_equal_prefill(cuda_lib):
    d = make((40, 40, 40), 4, 2, 128, 128, "f32", seed=12)
    want, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["s0"])
    s = d["s0"].clone()
    steps = {x: d[x].unflatten(0, (3, 40)).transpose(0, 1).contiguous() for x in ("q", "k", "v", "g")}
    outs = [kda.lin_decode_step(steps["q"][t], steps["k"][t], steps["v"][t], steps["g"][t], s) for t in range(40)]
    near(torch.stack(outs, 1).flatten(0, 1), np32(want), 1e-5, "out")
    near(s, np32(fin), 1e-5, "state")


def check_grads(got, ref, dtype):
    for name in ("dq", "dk", "dv", "dg"):
        assert got[name].dtype == DT[dtype]
        terms = 0.0
        if name == "dg" and ref["dg"].ndim == 1:
            size = np.abs(ref["dg_tokens"])
            terms = np.linalg.norm([size[t:t + 128].sum(0) for t in range(0, len(size), 128)])
        near(got[name], ref[name], TOL[DT[dtype]], name, room=TOL[DT[dtype]] * terms)
    near(got["ds0"], ref["ds0"], 2e-5 if dtype == "bf16" else 1e-5, "ds0")


@pytest.mark.parametrize("dtype,dk,dv", SHAPES)
@pytest.mark.parametrize("lengths", [(0, 5, 64, 130), (300, 1, 127), (777,)], ids=str)
def test_gradients_match_oracle(cuda_lib, dtype, dk, dv, lengths):
    seed = sum(lengths)
    d = make(lengths, 4, 2 if seed % 2 else 4, dk, dv, dtype, per_head=len(lengths) == 3, s0=len(lengths) != 1, seed=seed)
    got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], scale=0.5, initial_state=d["s0"],
                      d_final_state=d["dsf"] if len(lengths) > 1 else None, cu_seqlens_host=d["host"])
    ref = O.backward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], np32(d["dy"]), scale=0.5,
                     initial_state=np32(d["s0"]), d_final_state=np32(d["dsf"]) if len(lengths) > 1 else None)
    check_grads(got, ref, dtype)


def test_gradient_of_single_tokens_without_state(cuda_lib):
    """dg of a first token is exactly zero when there is no state to decay."""
    for dtype in DT:
        d = make((1, 1, 1), 4, 2, 64, 64, dtype, s0=False, seed=13)
        got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], d_final_state=d["dsf"])
        assert (got["dg"] == 0).all()
        ref = O.backward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], np32(d["dy"]),
                         d_final_state=np32(d["dsf"]))
        near(got["dk"], ref["dk"], TOL[DT[dtype]], "dk")


def test_gradient_is_the_derivative_of_the_forward(cuda_lib):
    """Along a random direction, (L(x + e) - L(x - e)) / 2 against the gradient, both from the kernels."""
    d = make((150, 41), 2, 1, 64, 64, "f32", seed=14)
    got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], scale=0.5, initial_state=d["s0"],
                      d_final_state=d["dsf"])
    gen = torch.Generator(device="cuda").manual_seed(15)

    def loss(x):
        o, fin = kda.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], d["cu"], scale=0.5, initial_state=x["s0"])
        return float((o.double() * d["dy"]).sum() + (fin.double() * d["dsf"]).sum())

    for key, name in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("s0", "ds0")):
        u = torch.randn(d[key].shape, generator=gen, device="cuda")
        e = 1e-3 if key == "g" else 1e-2
        slope = (loss({**d, key: d[key] + e * u}) - loss({**d, key: d[key] - e * u})) / (2 * e)
        want = float((got[name].double() * u).sum())
        # the loss is linear or nearly so in each input; its fp32 rounding over 2 e bounds the rest
        size = float(got[name].double().norm() * u.double().norm())
        assert abs(slope - want) <= 1e-3 * size, (key, slope, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_and_replayed(cuda_lib, dtype):
    """Forward, backward and a decode step in one graph, replayed on new values."""
    d = make((333, 50), 4, 2, 128, 128, dtype, seed=16)
    e = make((333, 50), 4, 2, 128, 128, dtype, seed=17)
    cur = {k: x.clone() if torch.is_tensor(x) else x for k, x in d.items()}
    state = cur["s0"].clone()

    def work():
        out, fin = kda.lin_chunk_fwd(cur["q"], cur["k"], cur["v"], cur["g"], cur["cu"], initial_state=cur["s0"])
        got = kda.lin_bwd(cur["q"], cur["k"], cur["v"], cur["g"], cur["dy"], cur["cu"], initial_state=cur["s0"],
                          cu_seqlens_host=cur["host"])
        dec = kda.lin_decode_step(cur["q"][:2], cur["k"][:2], cur["v"][:2], cur["g"][:2], state)
        return [out, fin, dec] + list(got.values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = work()
    for x in (e, d):
        for k in ("q", "k", "v", "g", "s0", "dy"):
            cur[k].copy_(x[k])
        state.copy_(x["s0"])
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        state.copy_(x["s0"])
        want = work()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once(cuda_lib):
    d = [make((900,), 4, 4, 128, 128, "bf16", seed=s) for s in (18, 19)]
    want = [kda.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"])[0] for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    for _ in range(4):
        got = []
        for x, s in zip(d, streams):
            ws = torch.empty(kda.lin_workspace_size(900, 1, 4, 4, 128, 128), dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            got.append((kda.lin_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["cu"], workspace=ws, stream=s)[0], ws))
        torch.cuda.synchronize()
        for (a, _), b in zip(got, want):
            assert torch.equal(a, b)


def test_bindings_refuse_other_layouts(cuda_lib):
    d = make((8,), 2, 2, 64, 64, "bf16", seed=20)
    bad = dict(q=d["q"].transpose(0, 1).contiguous().transpose(0, 1), k=d["k"][:4], v=d["v"].float(), g=d["g"].cpu())
    for name, t in bad.items():
        args = {**{x: d[x] for x in ("q", "k", "v", "g")}, name: t}
        with pytest.raises(ValueError):
            kda.lin_chunk_fwd(*args.values(), d["cu"])
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"].long())
    with pytest.raises(TypeError):
        kda.lin_chunk_fwd(*(d[x].half() for x in ("q", "k", "v", "g")), d["cu"])
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], cu_seqlens_host=[0, 4, 8])
    with pytest.raises(kda.KdaError):
        kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], cu_seqlens_host=[0, 4])
    with pytest.raises(ValueError):
        kda.lin_decode_step(d["q"], d["k"], d["v"], d["g"], torch.zeros(8, 2, 64, 64, device="cuda").bfloat16())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_layer_of_them(cuda_lib, dtype):
    """Linear attention, its per-head norm with the gate, and the residual with
    the next norm, forward and backward as a training step runs them, against
    fp64 autograd of the formulas on the same inputs."""
    H, D = 4, 64
    d = make((100, 29), H, 2, D, D, dtype, s0=False, seed=21)
    gen = torch.Generator().manual_seed(22)
    dt, T = DT[dtype], 129
    gate, x, dr, dh = (torch.randn(T, H * D, generator=gen).to(dt).cuda() for _ in range(4))
    w, wn = (1 + 0.1 * torch.randn(n, generator=gen).to(dt).cuda() for n in (D, H * D))

    kw1 = dict(post_weight=w, gate=gate.view(T, H, D), gate_logits=True)
    kw2 = dict(post_norm=False, residual=x, res_scale=0.5, pre_norm=True, pre_weight=wn)
    o, _ = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], scale=0.5)
    u, _ = kda.block_norm(o, **kw1)
    r, h = kda.block_norm(u.view(T, H * D), **kw2)
    b2 = kda.block_norm_bwd(dr, dh, u.view(T, H * D), **kw2)
    b1 = kda.block_norm_bwd(b2["dy"].view(T, H, D), None, o, **kw1)
    got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], b1["dy"], d["cu"], scale=0.5)

    names = ("q", "k", "v", "g")
    leaf = {n: d[n].double().cpu().requires_grad_() for n in names}
    leaf.update({n: t.double().cpu().requires_grad_() for n, t in dict(gate=gate, x=x, w=w, wn=wn).items()})
    q, k = (leaf[n].repeat_interleave(2, 1) for n in ("q", "k"))
    outs = []
    for a, b in ((0, 100), (100, 129)):
        G = leaf["g"][a:b].cumsum(0).T
        low = torch.ones(b - a, b - a, dtype=torch.bool).tril()
        Dm = torch.where(low, G[:, :, None] - G[:, None], -torch.inf).exp()
        A = torch.einsum("thd,shd->hts", 0.5 * q[a:b], k[a:b]) * Dm
        outs.append(torch.einsum("hts,shd->thd", A, leaf["v"][a:b]))
    ro = torch.cat(outs)
    rms = lambda t: t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    ru = rms(ro) * leaf["w"] * leaf["gate"].view(T, H, D).sigmoid()
    rr = leaf["x"] + 0.5 * ru.flatten(1)
    rh = rms(rr) * leaf["wn"]
    ref = dict(zip(leaf, torch.autograd.grad((rr, rh), list(leaf.values()), (dr.double().cpu(), dh.double().cpu()))))
    # a bf16 chain rounds every tensor on the way (o, u, dy twice: each 2^-8 / sqrt(3) at
    # most in the root mean square), on top of the single operator's 3.9e-3
    tol = 4 * TOL[dt]
    for name, t, e in (("r", r, rr), ("h", h, rh), ("dx", b2["dresidual"], ref["x"]), ("dwn", b2["dpre_weight"], ref["wn"]),
                       ("dw", b1["dpost_weight"], ref["w"]), ("dgate", b1["dgate"].flatten(1), ref["gate"]),
                       ("dq", got["dq"], ref["q"]), ("dk", got["dk"], ref["k"]), ("dv", got["dv"], ref["v"]),
                       ("dg", got["dg"], ref["g"])):
        near(t, e.detach().numpy(), tol, name)


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradients_of_rows_behind_the_last_sequence(cuda_lib, dtype, per_head):
    """They are zero in the binding's results and stay out of the sums."""
    d = make((100, 60), 4, 2, 64, 64, dtype, per_head=per_head, seed=23)
    cut = lambda x: x if x.dim() == 1 else x[:150].contiguous()  # noqa: E731
    cu = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    args = [d[x] for x in ("q", "k", "v", "g", "dy")]
    want = kda.lin_bwd(*(cut(x) for x in args), cu, initial_state=d["s0"])
    for x in args:
        if x.dim() > 1:
            x[150:] = float("nan")
    got = kda.lin_bwd(*args, cu, initial_state=d["s0"])
    for name in want:
        g = got[name]
        if g.shape != want[name].shape:
            assert (g[150:] == 0).all(), name
            g = g[:150]
        near(g, np32(want[name]), TOL[DT[dtype]], name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_workspace_reports_no_error(cuda_lib, dtype):
    d = make((300, 40), 2, 2, 64, 128, dtype, seed=24)
    ws = torch.full((kda.lin_workspace_size(340, 2, 2, 2, 64, 128, DT[dtype]),), 255, dtype=torch.uint8, device="cuda")
    kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], workspace=ws)
    assert kda.chunk_fwd_check(ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_no_tokens_at_all(cuda_lib, dtype):
    """Empty sequences only: states pass through, forward and backward."""
    d = make((0, 0, 0), 2, 1, 64, 128, dtype, per_head=True, seed=25)
    out, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["s0"])
    assert out.shape == (0, 2, 128) and torch.equal(fin, d["s0"])
    got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], initial_state=d["s0"], d_final_state=d["dsf"])
    assert torch.equal(got["ds0"], d["dsf"]) and (got["dg"] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_as_windows(cuda_lib, dtype):
    """Enough sequences and heads that a CTA takes a whole sequence when the host
    knows the lengths: the same results as through windows, and the oracle's."""
    lengths = (257, 0, 64, 500, 1, 130, 128, 300, 90, 411, 2, 350)
    d = make(lengths, 48, 24, 64, 64, dtype, seed=26)
    kw = dict(scale=0.5, initial_state=d["s0"])
    a = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], cu_seqlens_host=d["host"], **kw)
    b = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], **kw)
    for x, y, tol in zip(a, b, (TOL[DT[dtype]], 2e-5)):
        near(x, np32(y), tol, "by sequence")
    o, S = O.forward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], scale=0.5, initial_state=np32(d["s0"]))
    near(a[0], o, TOL[DT[dtype]], "out")
    near(a[1], S, 2e-5, "state")
    args = (d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"])
    a = kda.lin_bwd(*args, d_final_state=d["dsf"], cu_seqlens_host=d["host"], **kw)
    b = kda.lin_bwd(*args, d_final_state=d["dsf"], **kw)
    for name in a:
        near(a[name], np32(b[name]), 2e-5 if name == "ds0" else 2 * TOL[DT[dtype]], name)


def test_a_call_on_another_stream_keeps_its_memory(cuda_lib):
    """Workspace and results made inside a call on a given stream are not handed
    out to the current one before that stream has passed the call."""
    d = make((3000,), 8, 8, 128, 128, "bf16", seed=27)
    want, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["s0"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        out, s = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], initial_state=d["s0"], stream=side)
        junk = [torch.full((1 << 22,), float("nan"), device="cuda") for _ in range(4)]  # on the current stream
        side.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(s, fin)
        del junk, out, s


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [-5.0, -1.0, -0.05])
def test_dg_of_strong_and_weak_decays(cuda_lib, dtype, g):
    """Every head alike, so that no head with a long memory hides the others: with
    g = -5 dg is 150 times smaller than the terms q . dq and k . dk themselves."""
    d = make((300, 70), 2, 2, 64, 128, dtype, s0=False, seed=28)
    d["g"] = torch.full_like(d["g"], g)
    got = kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], scale=0.5)
    ref = O.backward(np32(d["q"]), np32(d["k"]), np32(d["v"]), np32(d["g"]), d["host"], np32(d["dy"]), scale=0.5)
    near(got["dg"], ref["dg"], TOL[DT[dtype]], "dg")
    assert (got["dg"][[0, 300]] == 0).all()


@pytest.mark.parametrize("where", ["all", "far"])
@pytest.mark.parametrize("per_head", [False, True])
def test_long_windows(cuda_lib, where, per_head):
    """Windows of 17 and 16 chunks, whose summaries leave out what the decays have
    forgotten: the state behind the last token and the gradient of the one before
    the first, against their sums in 64 bits.  far: only tokens at the far end have
    values, 1e30 of them, so that what remains of them is all there is.
    The exponents are sums of up to 33 chunks' decays, each rounded at 2^-19 at
    most (under 32 in absolute value, in powers of two): 33 x 2^-19 x ln 2 = 5e-5."""
    T, H, D = 4200, 74, 64
    gen = torch.Generator().manual_seed(31)
    randn = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16).cuda()  # noqa: E731
    q, k, v, dy = randn(T, H, D), randn(T, H, D), randn(T, H, D), randn(T, H, D)
    # from 1 (forgotten at once) down to nothing forgotten in the whole sequence
    slope = torch.logspace(0, -5, H).cuda()
    slope[-1] = 0.0
    g = (-slope if per_head else -slope * torch.rand(T, H, generator=gen).cuda()).to(torch.bfloat16)
    if where == "far":
        v[20:], dy[:T - 20] = 0, 0
        v[:20] *= 1e30
        dy[T - 20:] *= 1e30
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    o, S = kda.lin_chunk_fwd(q, k, v, g, cu)
    ds0 = kda.lin_bwd(q, k, v, g, dy, cu)["ds0"]
    gd = g.double().expand(T, H)
    through = gd.cumsum(0)
    want = torch.einsum("thk,th,thv->hkv", k.double(), (through[-1] - through).exp(), v.double())
    dwant = torch.einsum("thk,th,thv->hkv", q.double(), through.exp(), dy.double())
    for got, exact, what in ((S[0], want, "state"), (ds0[0], dwant, "ds0")):
        assert torch.isfinite(got).all()
        size = exact.abs().amax((1, 2))
        err = (got.double() - exact).norm(dim=(1, 2)) / exact.norm(dim=(1, 2)).clamp_min(1e-300)
        bad = (err > 6e-5) & (size > 1e-30)
        assert not bad.any(), f"{what}: heads {bad.nonzero().flatten().tolist()} off by {err[bad].tolist()}"
        assert (got.abs().amax((1, 2))[size < 1e-46] == 0).all(), what
    if where == "all":
        near(o[-1], np32(torch.einsum("hk,hkv->hv", q[-1].double(), want)), 1e-2, "last output")


def off_by(got, want):
    """||err||_2 / ||want||_2 on the device, for tensors too large to bring to the host."""
    assert torch.isfinite(got).all()
    return float((got.double() - want.double()).norm() / want.double().norm())


@pytest.mark.parametrize("lengths,H,Hk", [
    # a CTA runs whole sequences whose last chunk (the first one of the reversed passes) has one quarter of 32 tokens
    (tuple(128 * (3 * i % 11) + 1 + 5 * i % 32 for i in range(36)), 32, 4),
    # nothing but such chunks
    (tuple(1 + 7 * i % 32 for i in range(600)), 32, 32),
    # one, two and three quarters in turn
    (tuple(1 + 37 * i % 128 for i in range(700)), 16, 16)], ids=("tails", "short", "mixed"))
def test_short_chunks_of_large_batches(cuda_lib, lengths, H, Hk):
    """q, k, v and dy together beyond the size of the L2 cache, so that a chunk's
    loads arrive at different times: bf16 against the fp32 path on the same values
    (the oracle would take minutes), and against itself."""
    d = make(lengths, H, Hk, 128, 128, "bf16", seed=32)
    kw = dict(scale=0.5, initial_state=d["s0"], cu_seqlens_host=d["host"])
    args = [d[x] for x in ("q", "k", "v", "g")]
    ref = kda.lin_chunk_fwd(*(x.float() for x in args), d["cu"], **kw)
    rgrad = kda.lin_bwd(*(x.float() for x in args), d["dy"].float(), d["cu"], d_final_state=d["dsf"], **kw)
    first = None
    for _ in range(3):
        out, fin = kda.lin_chunk_fwd(*args, d["cu"], **kw)
        got = kda.lin_bwd(*args, d["dy"], d["cu"], d_final_state=d["dsf"], **kw)
        # (the fp32 results' own 1e-5 on top of the operator's tolerances)
        assert off_by(out, ref[0]) <= 4e-3 + 1e-5 and off_by(fin, ref[1]) <= 2e-5 + 1e-5
        for name in ("dq", "dk", "dv", "dg"):
            assert off_by(got[name], rgrad[name]) <= 4e-3 + 1e-5, name
        assert off_by(got["ds0"], rgrad["ds0"]) <= 2e-5 + 1e-5
        all_of = [out, fin, *got.values()]
        assert first is None or all(torch.equal(a, b) for a, b in zip(all_of, first))
        first = all_of


def long_work():
    """Some ten milliseconds for the current stream."""
    a = torch.randn(8192, 8192, device="cuda")
    for _ in range(10):
        a = a @ a * 1e-4
    return a


def on_a_side_stream(call):
    """call(stream), made while the current stream is busy and has freed memory of
    the results' sizes that it still writes, as a dict; and call(None), beforehand."""
    as_dict = lambda x: x if isinstance(x, dict) else dict(enumerate(x if isinstance(x, tuple) else (x,)))  # noqa: E731
    want = as_dict(call(None))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        busy = long_work()
        for t in [torch.empty_like(x) for x in want.values() if x is not None]:
            t.fill_(float("nan"))  # behind the long work; the memory goes back to the allocator here
        got = as_dict(call(side))
        side.synchronize()
        torch.cuda.synchronize()
        del busy
        for name, x in want.items():
            assert (x is None) == (got[name] is None) and (x is None or torch.equal(x, got[name])), name


@pytest.mark.parametrize("host", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_results_on_a_given_stream_wait_for_no_other(cuda_lib, dtype, host):
    """Nothing that the current stream has yet to do, the call's own fills among
    them, reaches the results of a call on another stream."""
    d = make((300, 50), 4, 2, 64, 64, dtype, seed=33)
    kw = dict(scale=0.5, initial_state=d["s0"], cu_seqlens_host=d["host"] if host else None)
    args = [d[x] for x in ("q", "k", "v", "g")]
    on_a_side_stream(lambda s: kda.lin_chunk_fwd(*args, d["cu"], stream=s, **kw))
    on_a_side_stream(lambda s: kda.lin_bwd(*args, d["dy"], d["cu"], d_final_state=d["dsf"], stream=s, **kw))
    gate, w = torch.randn_like(d["v"]), torch.ones(64, device="cuda", dtype=DT[dtype])
    norm = dict(post_weight=w, gate=gate, gate_logits=True, residual=d["dy"], pre_norm=True, pre_weight=w)
    on_a_side_stream(lambda s: kda.block_norm(d["v"], stream=s, **norm))
    on_a_side_stream(lambda s: kda.block_norm_bwd(d["dy"], gate, d["v"], stream=s, **norm))
    step = [x[:2].contiguous() for x in args]
    states = iter([d["s0"].clone() for _ in range(3)])  # one for each call
    on_a_side_stream(lambda s: kda.lin_decode_step(*step, next(states), stream=s))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_an_overflowing_sequence_leaves_its_neighbours_alone(cuda_lib, dtype):
    """Finite inputs whose state overflows, in sequences that cross windows: the
    sequence behind (in the gradient: before) them has the oracle's results."""
    d = make((1500, 1500), 2, 2, 64, 64, dtype, s0=False, seed=34)
    args = lambda: [d[x] for x in ("q", "k", "v", "g")]  # noqa: E731
    ref, S = O.forward(*(np32(x) for x in args()), d["host"], scale=0.5)
    rgrad = O.backward(*(np32(x) for x in args()), d["host"], np32(d["dy"]), scale=0.5)
    tol, stol = TOL[DT[dtype]], 2e-5 if dtype == "bf16" else 1e-5
    kept = {x: d[x].clone() for x in ("q", "k", "v", "dy")}
    d["k"][:1500], d["v"][:1500] = 1e25, 1e25
    for host in (None, d["host"]):
        out, fin = kda.lin_chunk_fwd(*args(), d["cu"], scale=0.5, cu_seqlens_host=host)
        assert not torch.isfinite(fin[0]).all()
        near(out[1500:], ref[1500:], tol, "out")
        near(fin[1], S[1], stol, "final state")
    d.update({x: t.clone() for x, t in kept.items()})
    d["q"][1500:], d["dy"][1500:] = 1e25, 1e25
    for host in (None, d["host"]):
        got = kda.lin_bwd(*args(), d["dy"], d["cu"], scale=0.5, cu_seqlens_host=host)
        assert not torch.isfinite(got["ds0"][1]).all()
        for name in ("dq", "dk", "dv", "dg"):
            near(got[name][:1500], rgrad[name][:1500], tol, name)
        near(got["ds0"][0], rgrad["ds0"][0], stol, "ds0")


@pytest.mark.parametrize("host", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_decays_are_not_hidden(cuda_lib, dtype, host):
    """A NaN log-decay is NaN in what depends on it, as in the single-token step,
    and nothing else."""
    d = make((400, 300), 2, 2, 64, 64, dtype, seed=35)
    args = [d[x] for x in ("q", "k", "v", "g")]
    kw = dict(scale=0.5, initial_state=d["s0"], cu_seqlens_host=d["host"] if host else None)
    want = (*kda.lin_chunk_fwd(*args, d["cu"], **kw), kda.lin_bwd(*args, d["dy"], d["cu"], **kw))
    t = 200
    d["g"][t, 1] = float("nan")
    out, fin = kda.lin_chunk_fwd(*args, d["cu"], **kw)
    got = kda.lin_bwd(*args, d["dy"], d["cu"], **kw)
    nan = lambda x: torch.isnan(x).all()  # noqa: E731
    assert nan(out[t:400, 1]) and nan(fin[0, 1]) and nan(got["dq"][t:400, 1])
    assert nan(got["dk"][:t, 1]) and nan(got["dv"][:t, 1]) and nan(got["dg"][t, 1]) and nan(got["ds0"][0, 1])
    out[t:400, 1], fin[0, 1] = want[0][t:400, 1], want[1][0, 1]
    assert torch.equal(out, want[0]) and torch.equal(fin, want[1])
    for name in want[2]:
        x, y = got[name], want[2][name]
        assert torch.equal(x[1:, 1], y[1:, 1]) and torch.equal(x[:, 0], y[:, 0]) if name == "ds0" else (
            torch.equal(x[400:], y[400:]) and torch.equal(x[:, 0], y[:, 0])), name
    s = d["s0"].clone()
    kda.lin_decode_step(*(x[:2].contiguous() for x in args[:3]), d["g"][t:t + 2].contiguous(), s)
    assert nan(s[0, 1]) and torch.isfinite(s[:, 0]).all()


def test_no_sequences_at_all(cuda_lib):
    """The gradient of a decay per head is a sum, which over nothing is zero."""
    d = make((), 4, 2, 64, 128, "bf16", per_head=True, seed=36)
    junk = torch.full((64, 4), float("nan"), device="cuda", dtype=torch.bfloat16)
    del junk
    out, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"], cu_seqlens_host=[0])
    assert out.shape == (0, 4, 128) and fin.shape == (0, 4, 64, 128)
    dg = torch.full((4,), 7.0, device="cuda", dtype=torch.bfloat16)
    lib, P = kda.load(), torch.Tensor.data_ptr
    ws = torch.empty(max(kda.lin_bwd_workspace_size(0, 0, 4, 2, 64, 128), 16), dtype=torch.uint8, device="cuda")
    st = lib.kda_lin_bwd(*[None] * 5, P(d["cu"]), None, 0, 0, 4, 2, 64, 128, kda.KDA_DTYPE_BF16, 1.0, kda.LIN_DECAY_PER_HEAD,
                         None, None, None, None, None, P(dg), None, P(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and (dg == 0).all()
    assert (kda.lin_bwd(d["q"], d["k"], d["v"], d["g"], d["dy"], d["cu"], cu_seqlens_host=[0])["dg"] == 0).all()


def test_fp32_writes_behind_strong_decays(cuda_lib):
    """A token at the end of a block of strong decays, the only one with a value:
    the state is k v^T, written as k (v e^-G) and renormalised by e^G, two
    exponentials within two half steps of 2^-24 and four products: 8 half steps."""
    T, H = 16, 64
    d = make((T,), H, H, 64, 64, "f32", s0=False, seed=37)
    d["g"] = torch.linspace(-2.45, -1.0, H, device="cuda").expand(T, H).contiguous()
    d["v"][:-1] = 0
    _, fin = kda.lin_chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["cu"])
    want = d["k"][-1].double()[:, :, None] * d["v"][-1].double()[:, None]
    assert ((fin[0].double() - want).abs() <= 8 * 2.0 ** -24 * want.abs()).all()


def test_fp32_decay_of_a_single_step(cuda_lib):
    """Nothing written: the state is S e^g, an exponential within two half steps of
    2^-24 and a product: 3 half steps."""
    N, H = 2, 64
    d = make((1,) * N, H, H, 64, 64, "f32", seed=38)
    d["g"] = torch.linspace(-80.0, 0.0, N * H, device="cuda").view(N, H).contiguous()
    d["k"].zero_()
    s = d["s0"].sign() * (d["s0"].abs() + 0.01)  # (so that e^-80 of it is a normal number)
    want = s.double() * d["g"].double().exp()[:, :, None, None]
    kda.lin_decode_step(d["q"], d["k"], d["v"], d["g"], s)
    assert ((s.double() - want).abs() <= 3 * 2.0 ** -24 * want.abs()).all()


def test_slow_decays_over_many_chunks(cuda_lib):
    """One window of 256 chunks per head, decays from forgetting at once to none,
    values of one sign, so that no rounding averages out.  The tensor cores
    truncate where they accumulate: a chunk's 16 products take up to 16 x 2^-23 of
    the state, and the sum of its decays is rounded by up to 2^-20 (in powers of
    two, under 32 in absolute value): 1.9e-6 + 2^-20 ln 2 = 2.6e-6 for each chunk
    that is remembered, on top of the parts' 2e-5."""
    T, H, D, block = 32768, 148, 64, 1024
    gen = torch.Generator(device="cuda").manual_seed(39)
    rand = lambda *s: torch.rand(*s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    k, v = rand(T, 1, D), rand(T, H, D)
    g = -torch.logspace(0, -6, H, device="cuda").bfloat16()
    g[-1] = 0
    _, fin = kda.lin_chunk_fwd(k, k, v, g, torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    gd, want = g.double(), torch.zeros(H, D, D, dtype=torch.float64, device="cuda")
    behind = (torch.arange(block - 1, -1, -1, device="cuda")[:, None] * gd).exp()
    for t in range(0, T, block):
        want *= (block * gd).exp()[:, None, None]
        want += torch.einsum("tk,thv->hkv", k[t:t + block, 0].double(), behind[:, :, None] * v[t:t + block].double())
    off = (fin[0].double() - want).norm(dim=(1, 2)) / want.norm(dim=(1, 2))
    remembered = (-(128 * gd).expm1()).clamp_min(128 / T).reciprocal()  # chunks: the sum of exp(128 g i), T / 128 at most
    assert (off <= 2e-5 + 2.6e-6 * remembered).all(), off.tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sequences_that_hold_none_of_the_tokens(cuda_lib, dtype):
    """Tokens, but all of them behind the last sequence, and every sequence empty."""
    d = make((70, 0, 130), 2, 1, 64, 128, dtype, per_head=True, seed=40)
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    out = torch.full_like(d["v"], 7.0)
    for x in ("q", "k", "v", "dy"):
        d[x].fill_(float("nan"))
    args = [d[x] for x in ("q", "k", "v", "g")]
    _, fin = kda.lin_chunk_fwd(*args, cu, initial_state=d["s0"], out=out)
    assert torch.equal(fin, d["s0"]) and (out == 7.0).all()
    got = kda.lin_bwd(*args, d["dy"], cu, initial_state=d["s0"], d_final_state=d["dsf"])
    assert torch.equal(got["ds0"], d["dsf"])
    assert all((got[x] == 0).all() for x in ("dq", "dk", "dv", "dg"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_state_in_place_of_whole_sequences(cuda_lib, dtype):
    """final_state = initial_state where a CTA takes a whole sequence."""
    d = make((257, 0, 64, 500, 1, 130, 128, 300, 90, 411, 2, 350), 48, 24, 64, 64, dtype, seed=41)
    args = [d[x] for x in ("q", "k", "v", "g")]
    want, fin = kda.lin_chunk_fwd(*args, d["cu"], initial_state=d["s0"], cu_seqlens_host=d["host"])
    s = d["s0"].clone()
    out, got = kda.lin_chunk_fwd(*args, d["cu"], initial_state=s, final_state=s, cu_seqlens_host=d["host"])
    assert got is s and torch.equal(out, want) and torch.equal(s, fin)


def test_two_streams_in_one_capture(cuda_lib):
    """Calls on the capturing stream and on one that it forks, side by side in a
    graph: the fills of the forked call are captured with it."""
    d, e = (make((333, 50), 4, 2, 64, 64, "bf16", seed=s) for s in (42, 43))
    args = lambda x: [x[n] for n in ("q", "k", "v", "g")]  # noqa: E731
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        side.wait_stream(main)
        got = kda.lin_bwd(*args(d), d["dy"], d["cu"], initial_state=d["s0"], stream=side)
        out = kda.lin_chunk_fwd(*args(e), e["cu"], initial_state=e["s0"])
        normed = kda.block_norm(d["v"], gate=d["dy"], gate_logits=True, stream=side)[0]
        main.wait_stream(side)
        return [*got.values(), *out, normed]

    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        want = [x.clone() for x in work()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=main):
            got = work()
    for _ in range(3):
        for x in got:
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
