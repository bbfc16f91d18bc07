"""Cases of the library's operators around linear attention with one decay per
head, and of the norms before and after a block, with their plain forms.

Two families:

  lin    per sequence and head, S_t = exp(g_t) S_{t-1} + k_t v_t^T,
         o_t = S_t^T (scale q_t): a prompt over packed sequences ("prefill"),
         one token per sequence ("decode"), and the gradient ("bwd").  q and k
         have Hk heads, each shared by H / Hk heads of v; g is one log-decay
         per token and head, or one per head ("per_head").
  norm   u = act(gate) * rmsnorm(y) * w_post, r = x + res_scale * u,
         h = rmsnorm(r) * w_pre, each part optional ("norm"), and its gradient
         ("norm_bwd").

`own` selects the library's kernels; without it the plain forms run, in torch
products, sums and exponentials in 32 bits (the log-decays are summed in 64).
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one short fp32 prompt: what a unit-sized call costs
        dict(name="prefill_tiny", kind="prefill", dtype="f32", lengths="256", H=2, Hk=2, dk=64, dv=64, s0=False, per_head=False),
        # two medium prompts, 16 heads: a training or prefill step of one layer
        dict(name="prefill_medium", kind="prefill", dtype="bf16", lengths="4096,4096", H=16, Hk=16, dk=128, dv=128, s0=False, per_head=False),
        # a batch of packed prompts of uneven lengths that continue from states; keys shared by pairs of heads
        dict(name="prefill_varlen", kind="prefill", dtype="bf16", lengths="5861,517,8011,3302,1,6977,4243,1290", H=32, Hk=16, dk=128, dv=128, s0=True, per_head=False),
        # one very long context, fixed decay per head
        dict(name="prefill_long", kind="prefill", dtype="bf16", lengths="131072", H=32, Hk=32, dk=128, dv=128, s0=False, per_head=True),
        # single-token step of a large batch: the state crosses HBM once each way
        dict(name="decode_batch", kind="decode", dtype="bf16", N=256, H=32, Hk=32, dk=128, dv=128, per_head=False),
        # single-token step of one request
        dict(name="decode_one", kind="decode", dtype="bf16", N=1, H=16, Hk=8, dk=128, dv=128, per_head=True),
        # the training step's gradient for two medium sequences
        dict(name="bwd_medium", kind="bwd", dtype="bf16", lengths="4096,4096", H=16, Hk=16, dk=128, dv=128, s0=False, per_head=False),
        # gradient of a packed fp32 batch with states, shared keys and an empty sequence
        dict(name="bwd_ragged", kind="bwd", dtype="f32", lengths="777,0,1501,64,3", H=8, Hk=4, dk=64, dv=128, s0=True, per_head=False),
        # the layer's output norm and gate, one row per token and head
        dict(name="norm_gate_heads", kind="norm", dtype="bf16", rows=8192 * 32, D=128, post=True, gate="logits", residual=False, pre=False),
        # the norms around a block for the tokens of one decode batch
        dict(name="norm_block_decode", kind="norm", dtype="bf16", rows=256, D=4096, post=True, gate="none", residual=True, pre=True),
        # gradient of the output norm and gate
        dict(name="norm_gate_heads_bwd", kind="norm_bwd", dtype="bf16", rows=8192 * 16, D=128, post=True, gate="logits", residual=False, pre=False),
        # gradient of the norms around a block for a training batch
        dict(name="norm_block_bwd", kind="norm_bwd", dtype="bf16", rows=8192, D=4096, post=True, gate="silu", residual=True, pre=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["prefill", "prefill", "decode", "bwd", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("norm", "norm_bwd"):
        D = rng.choice([64, 128, 128, _log_uniform(rng, 24, 8192), 8 * _log_uniform(rng, 8, 1024)])
        rows = _log_uniform(rng, 1, max(1, (1 << 24) // D))
        residual = rng.random() < 0.6
        return dict(kind=kind, dtype=dtype, rows=rows, D=D, post=residual is False or rng.random() < 0.7,
                    gate=rng.choice(["none", "given", "logits", "silu"]), residual=residual,
                    pre=residual and rng.random() < 0.8)
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    H = Hk * rng.choice([1, 1, 2, 4] if Hk <= 8 else [1, 2])
    dk, dv = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    per_head = rng.random() < 0.3
    if kind == "decode":
        return dict(kind=kind, dtype=dtype, N=_log_uniform(rng, 1, 256), H=H, Hk=Hk, dk=dk, dv=dv, per_head=per_head)
    N = rng.choice([1, 1, 2, 3, 5, 8])
    most = (65536 if kind == "prefill" else 8192) * 16 // (H * (2 if dtype == "f32" else 1))
    top = min(16384, max(2, most // N))
    lengths = [0 if rng.random() < 0.05 and N > 1 else _log_uniform(rng, 1, top) for _ in range(N)]
    if not any(lengths):
        lengths[0] = 33
    return dict(kind=kind, dtype=dtype, lengths=",".join(map(str, lengths)), H=H, Hk=Hk, dk=dk, dv=dv,
                s0=rng.random() < 0.5, per_head=per_head)


# ----------------------------------------------------------------- the inputs
def _lengths(case):
    return [int(x) for x in case["lengths"].split(",")]


def _decay_logits(H, device):
    # a spread of memories over the heads: about one token to about a thousand
    return -7.0 * torch.arange(H, device=device, dtype=torch.float32) / max(H - 1, 1)


def prepare(case, seed):
    dev, dt = "cuda", DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def chunk_plan(lengths, C, device):
        """Padded chunk layout of packed sequences: token index of each (chunk,
        row) and whether it exists; the sequence of each chunk; whether it is its
        sequence's last."""
        idx, seq = [], []
        at = 0
        for n, L in enumerate(lengths):
            for c in range(0, L, C):
                row = torch.arange(at + c, at + c + C)
                row[min(C, L - c):] = -1
                idx.append(row)
                seq.append(n)
            at += L
        idx = torch.stack(idx)
        return idx.clamp_min(0).to(device), (idx >= 0).to(device), torch.tensor(seq, device=device)

    s = dict(case=case)
    if case["kind"] in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        s["y"] = (randn(R, D) * 2.0).to(dt)
        s["w_post"] = (1.0 + 0.2 * randn(D)).to(dt) if case["post"] else None
        s["gate"] = None if case["gate"] == "none" else (randn(R, D).sigmoid() if case["gate"] == "given" else randn(R, D)).to(dt)
        s["x"] = randn(R, D).to(dt) if case["residual"] else None
        s["w_pre"] = (1.0 + 0.2 * randn(D)).to(dt) if case["pre"] else None
        s["scale"] = 0.35 if case["residual"] else 1.0
        if case["kind"] == "norm_bwd":
            s["dr"] = randn(R, D).to(dt)
            s["dh"] = randn(R, D).to(dt) if case["pre"] else None
        return s
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    lengths = None if case["kind"] == "decode" else _lengths(case)
    T = case["N"] if lengths is None else sum(lengths)
    N = case["N"] if lengths is None else len(lengths)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    s["q"], s["k"] = unit(randn(T, Hk, dk)).to(dt), unit(randn(T, Hk, dk)).to(dt)
    s["v"] = randn(T, H, dv).to(dt)
    bias = _decay_logits(H, dev)
    logits = bias if case["per_head"] else bias + randn(T, H)
    s["g"] = (-torch.nn.functional.softplus(logits)).to(dt)
    s["scale"] = 1.0 if lengths is None else 0.5
    if lengths is None:
        s["state"] = 0.02 * randn(N, H, dk, dv)
        return s
    s["s0"] = 0.02 * randn(N, H, dk, dv) if case["s0"] else None
    cu = [0]
    for L in lengths:
        cu.append(cu[-1] + L)
    s["cu"], s["cu_host"] = torch.tensor(cu, dtype=torch.int32, device=dev), cu
    s["plan"] = chunk_plan(lengths, 64 if T <= 32768 else 256, dev)
    if case["kind"] == "bwd":
        s["dy"] = randn(T, H, dv).to(dt)
        s["dsf"] = 0.5 * randn(N, H, dk, dv)
    return s


# ------------------------------------------------------------ the plain forms
def _plain_prefill(q, k, v, g, s0, plan, scale, N):
    """Chunks of the packed sequences side by side: the part of each chunk
    inside itself as a masked product, the state that enters each chunk as a
    decayed sum over the earlier chunks of its sequence."""
    idx, real, seq = plan
    H = v.shape[1]
    rep = H // q.shape[1]
    m = real[:, :, None, None]
    qc = (q[idx] * m).repeat_interleave(rep, 2).transpose(1, 2) * scale   # [nc, H, C, dk]
    kc = (k[idx] * m).repeat_interleave(rep, 2).transpose(1, 2)
    vc = (v[idx] * m).transpose(1, 2)
    gd = (g.double() if g.dim() == 2 else g.double().expand(v.shape[0], H))[idx] * real[:, :, None]
    G = gd.cumsum(1).transpose(1, 2)                                      # [nc, H, C], from the chunk's start
    C = G.shape[-1]
    low = torch.ones(C, C, dtype=torch.bool, device=G.device).tril()
    D = torch.where(low, G[..., :, None] - G[..., None, :], -torch.inf).exp().float()
    o = ((qc @ kc.transpose(-1, -2)) * D) @ vc
    total = G[..., -1]                                                    # [nc, H]
    Z = (kc * (total[..., None] - G).exp().float()[..., None]).transpose(-1, -2) @ vc
    before = seq[:, None] == seq[None, :]
    run = torch.where(before[..., None], total[None], 0.0)                # [c, c', H]
    nc = len(seq)
    earlier = torch.ones(nc, nc, dtype=torch.bool, device=G.device).tril(-1) & before
    start = torch.where(earlier[..., None], run, 0.0).sum(1)              # log-decay from the sequence's start to the chunk
    W = torch.where(earlier[..., None], start[:, None] - start[None] - total[None], -torch.inf).exp().float()
    S_in = torch.einsum("cdh,dhkv->chkv", W, Z)
    if s0 is not None:
        S_in = S_in + start.exp().float()[..., None, None] * s0[seq]
    o = o + (qc * G.exp().float()[..., None]) @ S_in
    S_out = S_in * total.exp().float()[..., None, None] + Z
    last = torch.ones(nc, dtype=torch.bool, device=G.device)
    last[:-1] = seq[1:] != seq[:-1]
    fin = torch.zeros(N, *Z.shape[1:], device=G.device) if s0 is None else s0
    fin = fin.index_copy(0, seq[last], S_out[last])                       # an empty sequence keeps its state
    out = torch.zeros(v.shape, device=G.device).index_put((idx[real],), o.transpose(1, 2)[real])
    return out, fin


def _plain_bwd(s):
    live = {n: s[n].float().requires_grad_() for n in ("q", "k", "v", "g")}
    N = len(s["cu_host"]) - 1
    dk, dv = s["q"].shape[-1], s["v"].shape[-1]
    s0 = torch.zeros(N, s["v"].shape[1], dk, dv, device=s["q"].device) if s["s0"] is None else s["s0"]
    s0 = s0.clone().requires_grad_()
    out, fin = _plain_prefill(live["q"], live["k"], live["v"], live["g"], s0, s["plan"], s["scale"], N)
    dt = s["q"].dtype
    got = torch.autograd.grad((out, fin), [live["q"], live["k"], live["v"], live["g"], s0],
                              (s["dy"].float(), s["dsf"]))
    return dict(dq=got[0].to(dt), dk=got[1].to(dt), dv=got[2].to(dt), dg=got[3].to(dt), ds0=got[4])


def _plain_decode(s):
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k, v = s["q"].float().repeat_interleave(rep, 1), s["k"].float().repeat_interleave(rep, 1), s["v"].float()
    a = s["g"].float().expand(v.shape[:2]).exp()
    S = s["state"]
    S.mul_(a[..., None, None]).add_(k[..., :, None] * v[..., None, :])
    out = (S * (s["scale"] * q)[..., :, None]).sum(-2)
    return out.to(s["q"].dtype), S


def _rms(x, w):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return n if w is None else n * w


def _plain_norm(case, y, w_post, gate, x, scale, w_pre):
    u = _rms(y, w_post) if case["post"] else y
    if gate is not None:
        z = gate
        u = u * {"given": z, "logits": z.sigmoid(), "silu": z * z.sigmoid()}[case["gate"]]
    r = u * scale if x is None else x + u * scale
    return r, (_rms(r, w_pre) if case["pre"] else None)


def _plain_norm_run(s):
    f = {n: None if s[n] is None else s[n].float() for n in ("y", "w_post", "gate", "x", "w_pre")}
    r, h = _plain_norm(s["case"], f["y"], f["w_post"], f["gate"], f["x"], s["scale"], f["w_pre"])
    dt = s["y"].dtype
    return r.to(dt), (None if h is None else h.to(dt))


def _plain_norm_bwd(s):
    names = [n for n in ("y", "w_post", "gate", "x", "w_pre") if s[n] is not None]
    f = {n: None if s[n] is None else s[n].float().requires_grad_() for n in ("y", "w_post", "gate", "x", "w_pre")}
    r, h = _plain_norm(s["case"], f["y"], f["w_post"], f["gate"], f["x"], s["scale"], f["w_pre"])
    outs, seeds = ((r,), (s["dr"].float(),)) if h is None else ((r, h), (s["dr"].float(), s["dh"].float()))
    got = dict(zip(names, torch.autograd.grad(outs, [f[n] for n in names], seeds)))
    dt = s["y"].dtype
    return {"d" + n: (x if n.startswith("w_") else x.to(dt)) for n, x in got.items()}


# ------------------------------------------------------------------- one pass
def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        from kda_linear_attention_fwd_b200 import kda
        if kind == "prefill":
            return kda.lin_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["cu"], scale=s["scale"],
                                     initial_state=s["s0"], cu_seqlens_host=s["cu_host"])
        if kind == "decode":
            return kda.lin_decode_step(s["q"], s["k"], s["v"], s["g"], s["state"], scale=s["scale"]), s["state"]
        if kind == "bwd":
            return kda.lin_bwd(s["q"], s["k"], s["v"], s["g"], s["dy"], s["cu"], scale=s["scale"],
                               initial_state=s["s0"], d_final_state=s["dsf"], cu_seqlens_host=s["cu_host"])
        args = dict(post_norm=case["post"], post_weight=s["w_post"], gate=s["gate"], gate_logits=case["gate"] == "logits",
                    gate_silu=case["gate"] == "silu", residual=s["x"], res_scale=s["scale"], pre_norm=case["pre"],
                    pre_weight=s["w_pre"], eps=EPS)
        if kind == "norm":
            return kda.block_norm(s["y"], **args)
        got = kda.block_norm_bwd(s["dr"], s["dh"], s["y"], **args)
        names = dict(dy="dy", dw_post="dpost_weight", dgate="dgate", dx="dresidual", dw_pre="dpre_weight")
        return {n: got[m] for n, m in names.items() if got[m] is not None}
    if kind == "prefill":
        out, fin = _plain_prefill(s["q"].float(), s["k"].float(), s["v"].float(), s["g"].float(), s["s0"], s["plan"],
                                  s["scale"], len(s["cu_host"]) - 1)
        return out.to(s["q"].dtype), fin
    if kind == "decode":
        return _plain_decode(s)
    if kind == "bwd":
        return _plain_bwd(s)
    return _plain_norm_run(s) if kind == "norm" else _plain_norm_bwd(s)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] in ("norm", "norm_bwd"):
        R, D = case["rows"], case["D"]
        ins = 1 + (case["gate"] != "none") + case["residual"]
        weights = case["post"] + case["pre"]
        if case["kind"] == "norm":
            return dict(bytes=R * D * e * (ins + 1 + case["pre"]) + weights * D * e, flops=R * D * (4 * weights + 6))
        return dict(bytes=R * D * e * (2 * ins + 1 + case["pre"]) + weights * D * (e + 4), flops=R * D * (12 * weights + 10))
    H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
    if case["kind"] == "decode":
        T = N = case["N"]
    else:
        T, N = sum(_lengths(case)), len(_lengths(case))
    g = (H if case["per_head"] else T * H) * e
    qk, vo, state = 2 * T * Hk * dk * e, T * H * dv * e, N * H * dk * dv * 4
    if case["kind"] == "decode":
        return dict(bytes=qk + 2 * vo + g + 2 * state, flops=5 * T * H * dk * dv)
    if case["kind"] == "prefill":
        return dict(bytes=qk + 2 * vo + g + state * (2 if case["s0"] else 1), flops=4 * T * H * dk * dv)
    # q, k, v, dy, g and the states in; dq, dk, dv, dg and dS0 out
    return dict(bytes=2 * qk + 3 * vo + 2 * g + state * (3 if case["s0"] else 2), flops=10 * T * H * dk * dv)


# ------------------------------------------------ the definitions, in 64 bits
def _exact_norm(case, s):
    d = {n: None if s.get(n) is None else s[n].double() for n in ("y", "w_post", "gate", "x", "w_pre", "dr", "dh")}
    y, z, c = d["y"], d["gate"], s["scale"]
    iy = 1.0 / ((y * y).mean(-1, keepdim=True) + EPS).sqrt() if case["post"] else 1.0
    wy = d["w_post"] if case["post"] else 1.0
    sg = None if z is None else 1.0 / (1.0 + (-z).exp())
    act = 1.0 if z is None else z if case["gate"] == "given" else sg if case["gate"] == "logits" else z * sg
    r = y * iy * wy * act * c + (d["x"] if d["x"] is not None else 0.0)
    ir = 1.0 / ((r * r).mean(-1, keepdim=True) + EPS).sqrt() if case["pre"] else None
    if case["kind"] == "norm":
        return r, (r * ir * d["w_pre"] if case["pre"] else None)
    out = {}
    dr = d["dr"]
    if case["pre"]:
        m = d["dh"] * d["w_pre"]
        rn = r * ir
        dr = dr + ir * (m - rn * (m * rn).mean(-1, keepdim=True))
        out["dw_pre"] = (d["dh"] * rn).sum(0)
    if d["x"] is not None:
        out["dx"] = dr
    du = dr * c
    yn = y * iy
    if z is not None:
        slope = 1.0 if case["gate"] == "given" else sg * (1 - sg) if case["gate"] == "logits" else sg * (1 + z * (1 - sg))
        out["dgate"] = du * yn * wy * slope
    dn = du * act
    if case["post"]:
        out["dw_post"] = (dn * yn).sum(0)
        m = dn * wy
        out["dy"] = iy * (m - yn * (m * yn).mean(-1, keepdim=True))
    else:
        out["dy"] = dn
    return out


def exact(case, seed):
    s = prepare(case, seed)

    def by_step(x, lengths):
        """[T, ...] packed -> [N, longest, ...] in 64 bits, zero behind each end."""
        out = x.new_zeros(len(lengths), max(lengths), *x.shape[1:], dtype=torch.float64)
        at = 0
        for n, L in enumerate(lengths):
            out[n, :L] = x[at:at + L]
            at += L
        return out

    def packed(x, lengths):
        return torch.cat([x[n, :L] for n, L in enumerate(lengths)])

    def exact_lin():
        lengths = _lengths(case)
        H, rep, T = case["H"], case["H"] // case["Hk"], sum(lengths)
        q = by_step(s["q"].double().repeat_interleave(rep, 1) * s["scale"], lengths)
        k = by_step(s["k"].double().repeat_interleave(rep, 1), lengths)
        v = by_step(s["v"].double(), lengths)
        a = by_step(s["g"].double().expand(T, H), lengths).exp()   # 1 behind each end
        N, L = v.shape[:2]
        S = torch.zeros(N, H, case["dk"], case["dv"], dtype=torch.float64, device=v.device)
        if s["s0"] is not None:
            S += s["s0"]
        if case["kind"] == "prefill":
            o = torch.empty_like(v)
            for t in range(L):
                S = torch.addcmul(S * a[:, t, :, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
                o[:, t] = (q[:, t, :, None, :] @ S)[:, :, 0]
            return packed(o, lengths), S
        do = by_step(s["dy"].double(), lengths)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        for t in range(L):
            S = torch.addcmul(S * a[:, t, :, None, None], k[:, t, :, :, None], v[:, t, :, None, :])
            dq[:, t] = (S @ do[:, t, :, :, None])[..., 0]
        B = s["dsf"].double()
        tail = (S * B).sum((-1, -2))                                # <S, dL/dS> behind the last token
        for t in reversed(range(L)):
            B = torch.addcmul(B, q[:, t, :, :, None], do[:, t, :, None, :])
            dk[:, t] = (B @ v[:, t, :, :, None])[..., 0]
            dv[:, t] = (k[:, t, :, None, :] @ B)[:, :, 0]
            B = B * a[:, t, :, None, None]
        # <a_t S_{t-1}, dL/dS_t> from the two products that change <S, dL/dS> on the way back
        steps = (q * dq).sum(-1) - (k * dk).sum(-1)
        dg = steps.flip(1).cumsum(1).flip(1) + tail[:, None]
        shared = lambda x: packed(x, lengths).unflatten(1, (case["Hk"], rep)).sum(2)  # noqa: E731
        dg = packed(dg, lengths)
        return dict(dq=shared(dq * s["scale"]), dk=shared(dk), dv=packed(dv, lengths),
                    dg=dg.sum(0) if case["per_head"] else dg, ds0=B)

    if case["kind"] in ("norm", "norm_bwd"):
        return _exact_norm(case, s)
    if case["kind"] == "decode":
        rep = case["H"] // case["Hk"]
        q, k = s["q"].double().repeat_interleave(rep, 1), s["k"].double().repeat_interleave(rep, 1)
        S = torch.empty(s["state"].shape, dtype=torch.float64, device="cuda")
        o = torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
        a = s["g"].double().expand(case["N"], case["H"]).exp()
        for n in range(case["N"]):
            S[n] = a[n, :, None, None] * s["state"][n].double() + k[n, :, :, None] * s["v"][n].double()[:, None, :]
            o[n] = torch.einsum("hkv,hk->hv", S[n], q[n] * s["scale"])
        return o, S
    return exact_lin()
