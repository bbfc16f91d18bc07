"""The norms around a block (kda_block_norm, kda_block_norm_bwd) on the GPU
against the fp64 oracle.

Tolerances, as ||err||_2 / ||ref||_2: bf16 results 2.4e-3 (one rounding: at
most 2^-8 / sqrt(3) = 2.3e-3 in the root mean square), fp32 results 2e-6
(some 30 half steps of 2^-24: sums over a row, a reciprocal root, an
exponential), fp32 sums over the rows 1e-5.  dy = iy (m - yn mean(m yn)) is a
difference whose terms cancel when a row's own direction dominates m (at D = 1
down to eps / (y^2 + eps) of either): the second term is a projection of the
first, so neither exceeds ||iy m||, each is computed to a few 2^-24 of itself,
and the error is a few 2^-24 of ||iy m|| however small the difference is.  So
dy may be off by its tolerance of ||dy|| plus the fp32 one of ||iy m||.
"""
import numpy as np
import pytest
import torch

from kda_linear_attention_fwd_b200 import kda
from oracle import linear as O
from parity import np32

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {"bf16": 2.4e-3, "f32": 2e-6}


def near(got, want, tol, what, room=0.0):
    a, e = np32(got).astype(np.float64), np.asarray(want, np.float64).reshape(got.shape)
    assert np.isfinite(a).all(), f"{what}: not finite"
    off = max(np.linalg.norm(a - e) - room, 0.0) / max(np.linalg.norm(e), 1e-30) if e.size else 0.0
    assert off <= tol, f"{what}: relative error {off:.2e} > {tol:.1e}"


def make(R, D, dtype, act, post, residual, pre, weights=True, seed=0):
    gen = torch.Generator().manual_seed(seed + R + D)
    randn = lambda *s: torch.randn(*s, generator=gen).to(DT[dtype]).cuda()  # noqa: E731
    d = dict(y=2 * randn(R, D), gate=None if act is None else randn(R, D), residual=randn(R, D) if residual else None,
             post_weight=randn(D) if post and weights else None, pre_weight=randn(D) if pre and weights else None)
    kw = dict(post_norm=post, pre_norm=pre, res_scale=0.4)
    return d, kw, randn(R, D), randn(R, D) if pre else None


def both(d, kw, act, dr, dh, dtype, eps=1e-6):
    t = {k: x for k, x in d.items() if k != "y"}
    gate = dict(gate_logits=act == "logits", gate_silu=act == "silu")
    ref_in = {k: np32(x) for k, x in t.items()}
    out, normed = kda.block_norm(d["y"], **t, **kw, **gate, eps=eps)
    ro, rn = O.block_norm(np32(d["y"]), **ref_in, **kw, act=act or "given", eps=eps)
    near(out, ro, TOL[dtype], "out")
    assert (normed is None) == (rn is None)
    if rn is not None:
        near(normed, rn, TOL[dtype], "normed")
    got = kda.block_norm_bwd(dr, dh, d["y"], **t, **kw, **gate, eps=eps)
    ref = O.block_norm_backward(np32(dr), np32(dh), np32(d["y"]), **ref_in, **kw, act=act or "given", eps=eps)
    for name in ("dy", "dgate", "dresidual", "dpost_weight", "dpre_weight"):
        if got[name] is None:
            continue
        want = ref[name] if ref[name] is not None else np.zeros(got[name].shape)
        near(got[name], want, 1e-5 if name.endswith("weight") else TOL[dtype], name,
             room=TOL["f32"] * np.linalg.norm(ref["dy_term"]) if name == "dy" else 0.0)
    return out, normed, got


KINDS = [("logits", True, False, False), ("silu", True, True, True), ("given", False, True, True),
         (None, True, True, True), (None, True, False, False), (None, False, True, False)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", KINDS, ids=str)
@pytest.mark.parametrize("R,D", [(1, 128), (300, 128), (5, 64), (33, 4096), (7, 1000)])
def test_matches_oracle(cuda_lib, dtype, kind, R, D):
    act, post, residual, pre = kind
    d, kw, dr, dh = make(R, D, dtype, act, post, residual, pre)
    both(d, kw, act, dr, dh, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 2, 7, 24, 129, 520, 1023, 2055, 4097, 8192, 8200, 16383, 16384])
def test_row_lengths(cuda_lib, dtype, D):
    """Every split of a row over threads, whole and single-element vectors."""
    d, kw, dr, dh = make(3, D, dtype, "silu", True, True, True)
    both(d, kw, "silu", dr, dh, dtype, eps=1e-3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(cuda_lib, dtype):
    """More rows than one wave of CTAs holds, an odd number of them."""
    d, kw, dr, dh = make(20011, 128, dtype, "logits", True, False, False)
    both(d, kw, "logits", dr, dh, dtype)


def test_without_weights(cuda_lib):
    d, kw, dr, dh = make(9, 256, "f32", None, True, True, True, weights=False)
    _, _, got = both(d, kw, None, dr, dh, "f32")
    assert got["dpost_weight"] is None and got["dpre_weight"] is None


def test_only_one_upstream_gradient(cuda_lib):
    d, kw, dr, dh = make(6, 192, "f32", "logits", True, True, True)
    both(d, kw, "logits", dr, None, "f32")
    both(d, kw, "logits", None, dh, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zero_and_huge_rows(cuda_lib, dtype):
    """A row of zeros stays zero; large values do not overflow the row sums."""
    d, kw, dr, dh = make(4, 128, dtype, "silu", True, False, False)
    d["y"][1] = 0
    d["y"][2] = 1e15
    d["gate"][3] = -200.0
    out, _, got = both(d, kw, "silu", dr, dh, dtype)
    assert (out[1] == 0).all()


@pytest.mark.parametrize("dtype,off", [("bf16", 0), ("bf16", 8), ("bf16", 3), ("f32", 1)])
def test_strided_rows(cuda_lib, dtype, off):
    """Inputs that are column slices of a wider tensor, aligned and not."""
    d, kw, dr, dh = make(17, 128, dtype, "logits", True, True, True)
    wide = torch.randn(17, 3 * 128 + 16, device="cuda").to(DT[dtype])
    for i, name in enumerate(("y", "gate", "residual")):
        view = wide[:, i * 128 + off:(i + 1) * 128 + off]
        view.copy_(d[name])
        d[name] = view
    both(d, kw, "logits", dr, dh, dtype)


def test_in_place_on_the_residual(cuda_lib):
    d, kw, _, _ = make(50, 512, "bf16", None, True, True, True)
    t = {k: x for k, x in d.items() if k not in ("y", "residual")}
    out, normed = kda.block_norm(d["y"], **t, **kw, residual=d["residual"])
    x, y = d["residual"].clone(), d["y"].clone()
    o2, n2 = kda.block_norm(y, **t, **kw, residual=x, out=x, normed=y)
    assert o2 is x and n2 is y and torch.equal(x, out) and torch.equal(y, normed)


def test_leading_shapes_and_no_rows(cuda_lib):
    y = torch.randn(3, 5, 64, device="cuda")
    out, normed = kda.block_norm(y)
    near(out, O.block_norm(np32(y).reshape(15, 64))[0], TOL["f32"], "out")
    assert out.shape == y.shape and normed is None
    e = torch.empty(0, 64, device="cuda")
    assert kda.block_norm(e, pre_norm=True)[1].shape == (0, 64)
    w = torch.ones(64, device="cuda")
    got = kda.block_norm_bwd(e, None, e, post_weight=w)
    assert (got["dpost_weight"] == 0).all()


def test_deterministic_and_captured(cuda_lib):
    d, kw, dr, dh = make(4000, 256, "bf16", "silu", True, True, True)
    t = {k: x for k, x in d.items() if k != "y"}
    run = lambda: list(kda.block_norm(d["y"], **t, **kw, gate_silu=True)) + list(  # noqa: E731
        kda.block_norm_bwd(dr, dh, d["y"], **t, **kw, gate_silu=True).values())
    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = run()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_bindings_refuse(cuda_lib):
    y = torch.randn(4, 64, device="cuda")
    for kw in (dict(gate=y[:, :32]), dict(gate=y.bfloat16()), dict(residual=y.t().contiguous().t()),
               dict(post_weight=torch.ones(32, device="cuda")), dict(gate=y, gate_logits=True, gate_silu=True),
               dict(post_norm=False, post_weight=torch.ones(64, device="cuda")),
               dict(pre_weight=torch.ones(64, device="cuda")), dict(normed=y), dict(out=y[:2])):
        with pytest.raises((ValueError, kda.KdaError)):
            kda.block_norm(y, **kw)
    with pytest.raises(ValueError):
        kda.block_norm_bwd(None, None, y)
    with pytest.raises(TypeError):
        kda.block_norm(y.half())


@pytest.mark.parametrize("act", ["logits", "silu"])
def test_gates_of_fp32_rows_are_fp32(cuda_lib, act):
    """Element by element, without a norm: logistic(z) = 1 / (1 + exp(-z)) from an
    exponential and a reciprocal within two half steps of 2^-24 each and a sum (one),
    and up to two products: 7 half steps, 8 in the slope's sum."""
    z = torch.linspace(-87.0, 87.0, 4096, device="cuda").view(2, 2048)
    y = torch.linspace(0.5, 2.0, 4096, device="cuda").view(2, 2048)
    kw = dict(post_norm=False, gate=z, gate_logits=act == "logits", gate_silu=act == "silu")
    out, _ = kda.block_norm(y, **kw)
    got = kda.block_norm_bwd(torch.ones_like(y), None, y, **kw)
    zd, yd = z.double(), y.double()
    s = zd.sigmoid()
    rest = (-zd).sigmoid()  # 1 - s
    value, slope = (s, s * rest) if act == "logits" else (zd * s, s * (1 + zd * rest))
    near_each = lambda a, e, n, room=0.0: ((a.double() - e).abs() - room <= n * 2.0 ** -24 * e.abs()).all()  # noqa: E731
    assert near_each(out, yd * value, 7)
    assert near_each(got["dy"], value, 7)
    # 1 - s cancels for large z: it is off by up to four half steps of s, and the silu's z (1 - s) by z of them
    assert near_each(got["dgate"], yd * slope, 8, (yd * s * (4 * (zd.abs() + 1 if act == "silu" else 1)) * 2.0 ** -24))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gates_at_the_ends(cuda_lib, dtype):
    """Closed and open gates, beyond what an exponential holds, and NaN."""
    ends = [-float("inf"), -3e38, -1e30, -200.0, 200.0, 1e30, 3e38, float("inf"), float("nan")]
    z = torch.tensor(ends, device="cuda").to(DT[dtype]).repeat(16).view(2, 72)
    y = torch.full_like(z, 2.0)
    out, _ = kda.block_norm(y, post_norm=False, gate=z, gate_logits=True)
    want = torch.tensor([0.0] * 4 + [2.0] * 4, device="cuda").to(DT[dtype])
    assert torch.equal(out.view(-1, 9)[:, :8], want.expand(16, 8)) and torch.isnan(out.view(-1, 9)[:, 8]).all()
    got = kda.block_norm_bwd(torch.ones_like(y), None, y, post_norm=False, gate=z, gate_logits=True)
    assert (got["dgate"].view(-1, 9)[:, :8] == 0).all() and torch.equal(got["dy"].view(-1, 9)[:, :8], want.expand(16, 8) / 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,D", [(15001, 256), (4001, 1000), (1003, 2304), (1000, 4096), (401, 2055), (1001, 5120), (910, 8192),
                                 (330, 9000), (310, 16384), (950, 4097)])
def test_several_rows_per_cta(cuda_lib, dtype, R, D):
    """Two or more rows for each group of threads, in every split of a row, of one warp, of
    several and with several vectors per thread: the loops over rows, with what
    they request ahead."""
    d, kw, dr, dh = make(R, D, dtype, "silu", True, True, True)
    both(d, kw, "silu", dr, dh, dtype, eps=1e-3)
    kw.update(pre_norm=False)
    d.update(pre_weight=None, residual=None)
    both(d, kw, "logits", dr, None, dtype, eps=1e-3)


def test_single_rows_and_scalars(cuda_lib):
    """A tensor of one dimension is one row; a strided one or a scalar is refused as such."""
    y = torch.randn(64, device="cuda")
    out, normed = kda.block_norm(y, pre_norm=True)
    assert out.shape == normed.shape == (64,)
    near(out[None], O.block_norm(np32(y)[None])[0], TOL["f32"], "out")
    for bad in (y[::2], y[0]):
        with pytest.raises(ValueError):
            kda.block_norm(bad)
        with pytest.raises(ValueError):
            kda.block_norm_bwd(bad, None, bad)
