"""Linear attention with one decay per head and the block norms without a GPU:
the oracle against closed forms and differences, and the C ABI's refusals."""
import ctypes

import numpy as np
import pytest

from kda_linear_attention_fwd_b200 import build, kda
from oracle import linear as O

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, -1, -2, -3, -4
BF16, F32 = 1, 0
A = 0x100000  # a 16-byte aligned fake device address; never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kda.load()


def _inputs(T, H, Hk, dk, dv, N, per_head, seed=0):
    rng = np.random.default_rng(seed)
    return dict(q=rng.standard_normal((T, Hk, dk)), k=rng.standard_normal((T, Hk, dk)),
                v=rng.standard_normal((T, H, dv)), g=-rng.exponential(0.5, (H,) if per_head else (T, H)),
                s0=rng.standard_normal((N, H, dk, dv)))


def test_oracle_is_the_decayed_sum():
    """o_t = sum_{s <= t} exp(G_t - G_s) (scale q_t . k_s) v_s, with no state."""
    d = _inputs(9, 4, 2, 3, 5, 1, False)
    o, fin = O.forward(d["q"], d["k"], d["v"], d["g"], [0, 9], scale=0.5)
    G = d["g"].cumsum(0)
    for h in range(4):
        w = np.tril(np.exp(G[:, None, h] - G[None, :, h])) * (0.5 * d["q"][:, h // 2] @ d["k"][:, h // 2].T)
        np.testing.assert_allclose(o[:, h], w @ d["v"][:, h], rtol=1e-12, atol=1e-12)
        last = (np.exp(G[-1, h] - G[:, h])[:, None] * d["k"][:, h // 2]).T @ d["v"][:, h]
        np.testing.assert_allclose(fin[0, h], last, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("per_head", [False, True])
def test_oracle_gradient_against_differences(per_head):
    cu = [0, 4, 4, 7]
    d = _inputs(7, 2, 1, 3, 2, 3, per_head, seed=1)
    rng = np.random.default_rng(2)
    dy, dsf = rng.standard_normal(d["v"].shape), rng.standard_normal(d["s0"].shape)

    def loss(x):
        o, fin = O.forward(x["q"], x["k"], x["v"], x["g"], cu, scale=0.7, initial_state=x["s0"])
        return (dy * o).sum() + (dsf * fin).sum()

    got = O.backward(d["q"], d["k"], d["v"], d["g"], cu, dy, scale=0.7, initial_state=d["s0"], d_final_state=dsf)
    for name, key in [("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("ds0", "s0")]:
        diff = np.zeros_like(d[key])
        for i in np.ndindex(*d[key].shape):
            e = 1e-6
            hi, lo = ({**d, key: d[key].copy()} for _ in range(2))
            hi[key][i] += e
            lo[key][i] -= e
            diff[i] = (loss(hi) - loss(lo)) / (2 * e)
        np.testing.assert_allclose(got[name], diff, rtol=1e-6, atol=1e-7)


@pytest.mark.parametrize("act,post,residual,pre", [("given", True, True, True), ("logits", True, False, False),
                                                   ("silu", False, True, True), (None, True, True, False)])
def test_oracle_norm_gradient_against_differences(act, post, residual, pre):
    rng = np.random.default_rng(3)
    d = dict(y=rng.standard_normal((3, 5)), gate=None if act is None else rng.standard_normal((3, 5)),
             residual=rng.standard_normal((3, 5)) if residual else None,
             post_weight=rng.standard_normal(5) if post else None, pre_weight=rng.standard_normal(5) if pre else None)
    kw = dict(post_norm=post, pre_norm=pre, act=act or "given", res_scale=0.6, eps=1e-3)
    dr, dh = rng.standard_normal((3, 5)), rng.standard_normal((3, 5)) if pre else None

    def loss(x):
        r, h = O.block_norm(x["y"], **{k: x[k] for k in x if k != "y"}, **kw)
        return (dr * r).sum() + ((dh * h).sum() if pre else 0.0)

    got = O.block_norm_backward(dr, dh, d["y"], **{k: d[k] for k in d if k != "y"}, **kw)
    for key in d:
        if d[key] is None:
            continue
        diff = np.zeros_like(d[key])
        for i in np.ndindex(*d[key].shape):
            hi, lo = ({**d, key: d[key].copy()} for _ in range(2))
            hi[key][i] += 1e-6
            lo[key][i] -= 1e-6
            diff[i] = (loss(hi) - loss(lo)) / 2e-6
        np.testing.assert_allclose(got["d" + key], diff, rtol=1e-6, atol=1e-7)


def host(xs):
    arr = (ctypes.c_int32 * len(xs))(*xs)
    return ctypes.cast(arr, ctypes.c_void_p)


def fwd(lib, **kw):
    a = dict(q=A, k=A, v=A, g=A, out=A, cu=A, cu_host=None, N=1, T=16, H=2, Hk=1, dk=64, dv=64, dtype=BF16,
             scale=1.0, flags=0, s0=None, s1=None, ws=A, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return lib.kda_lin_chunk_fwd(*a.values())


def test_lin_fwd_refusals(lib):
    assert fwd(lib, N=0, T=0) == OK
    assert fwd(lib, N=0) == INVALID
    for bad in (dict(N=-1), dict(T=-1), dict(H=0), dict(Hk=0), dict(Hk=3), dict(H=3, Hk=2), dict(flags=2),
                dict(q=None), dict(out=None), dict(cu=None), dict(cu_host=host([0, 15])),
                dict(N=2, cu_host=host([0, 17, 16])), dict(s0=A, s1=A + 256)):
        assert fwd(lib, **bad) == INVALID, bad
    for bad in (dict(dk=96), dict(dv=32), dict(dtype=2)):
        assert fwd(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=A + 2), dict(v=A + 8), dict(out=A + 8), dict(g=A + 1), dict(cu=A + 2), dict(s0=A + 4),
                dict(s1=A + 8), dict(ws=A + 8)):
        assert fwd(lib, **bad) == ALIGN, bad
    need = lib.kda_lin_chunk_fwd_workspace_size(16, 1, 2, 1, 64, 64, BF16)
    assert need > 0 and fwd(lib, ws_bytes=need - 1) == WORKSPACE and fwd(lib, ws=None) == WORKSPACE
    assert fwd(lib, s0=A, s1=A, ws=None) == WORKSPACE  # in place is accepted
    f = lib.kda_lin_chunk_fwd_workspace_size
    assert f(-1, 1, 1, 1, 64, 64, BF16) == 0 and f(16, 1, 3, 2, 64, 64, BF16) == 0 and f(16, 1, 1, 1, 96, 64, F32) == 0


def test_lin_decode_refusals(lib):
    def dec(**kw):
        a = dict(q=A, k=A, v=A, g=A, out=A, state=A, N=2, H=2, Hk=1, dk=64, dv=64, dtype=F32, scale=1.0, flags=0,
                 stream=None)
        a.update(kw)
        return lib.kda_lin_decode_step(*a.values())
    assert dec(N=0) == OK
    for bad in (dict(N=-1), dict(Hk=5), dict(flags=-1), dict(state=None), dict(g=None)):
        assert dec(**bad) == INVALID, bad
    assert dec(dk=32) == UNSUPPORTED and dec(dtype=9) == UNSUPPORTED
    assert dec(state=A + 8) == ALIGN and dec(k=A + 4) == ALIGN and dec(g=A + 2) == ALIGN


def test_lin_bwd_refusals(lib):
    need = lib.kda_lin_bwd_workspace_size(16, 1, 2, 1, 64, 64)

    def bwd(**kw):
        a = dict(q=A, k=A, v=A, g=A, dy=A, cu=A, cu_host=None, N=1, T=16, H=2, Hk=1, dk=64, dv=64, dtype=BF16,
                 scale=1.0, flags=0, s0=None, dsf=None, dq=A, dk_=A, dv_=A, dg=A, ds0=None, ws=A, ws_bytes=need,
                 stream=None)
        a.update(kw)
        return lib.kda_lin_bwd(*a.values())
    assert need > 0 and bwd(N=0, T=0) == OK
    for bad in (dict(dy=None), dict(dq=None), dict(dg=None), dict(cu=None), dict(flags=4), dict(Hk=4),
                dict(cu_host=host([0, 3])), dict(s0=A, ds0=A), dict(dsf=A, ds0=A + 16)):
        assert bwd(**bad) == INVALID, bad
    for bad in (dict(dq=A + 2), dict(dg=A + 1), dict(ds0=A + 4), dict(dy=A + 8)):
        assert bwd(**bad) == ALIGN, bad
    assert bwd(ws=None) == WORKSPACE and bwd(ws_bytes=need - 1) == WORKSPACE
    assert bwd(dk=16) == UNSUPPORTED


def test_norm_refusals(lib):
    def norm(**kw):
        a = dict(y=A, ys=64, wp=None, gate=None, gs=0, x=None, xs=0, wn=None, out=A, normed=None, rows=4, D=64,
                 dtype=BF16, c=1.0, eps=1e-6, flags=1, stream=None)
        a.update(kw)
        return lib.kda_block_norm(*a.values())
    assert norm(rows=0) == OK
    for bad in (dict(rows=-1), dict(D=0), dict(flags=16), dict(flags=12), dict(eps=-1.0), dict(eps=float("nan")),
                dict(y=None), dict(out=None), dict(ys=63), dict(gate=A, gs=10), dict(x=A, xs=8), dict(normed=A),
                dict(flags=3), dict(flags=0, wp=A), dict(wn=A)):
        assert norm(**bad) == INVALID, bad
    assert norm(dtype=4) == UNSUPPORTED and norm(D=16385, ys=16385) == UNSUPPORTED
    assert norm(y=A + 1) == ALIGN and norm(wp=A + 1) == ALIGN and norm(dtype=F32, out=A + 2) == ALIGN

    need = lib.kda_block_norm_bwd_workspace_size(4, 64, BF16)

    def bwd(**kw):
        a = dict(dout=A, dn=None, y=A, ys=64, wp=A, gate=A, gs=64, x=A, xs=64, wn=A, dy=A, dgate=A, dx=A, dwp=A,
                 dwn=A, rows=4, D=64, dtype=BF16, c=1.0, eps=1e-6, flags=3, ws=A, ws_bytes=need, stream=None)
        a.update(kw)
        return lib.kda_block_norm_bwd(*a.values())
    assert need > 0
    for bad in (dict(dout=None), dict(dy=None), dict(gate=None), dict(x=None), dict(flags=2), dict(flags=1),
                dict(wp=None), dict(ys=3)):
        assert bwd(**bad) == INVALID, bad
    assert bwd(ws=None) == WORKSPACE and bwd(ws_bytes=need - 1) == WORKSPACE
    assert bwd(dwp=A + 2) == ALIGN and bwd(dy=A + 1) == ALIGN


def test_bindings_refuse_what_the_kernels_cannot_read():
    import torch
    x, g = torch.zeros(4, 2, 64), torch.zeros(4, 2)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.lin_chunk_fwd(x, x, x, g, cu)
    with pytest.raises(ValueError):
        kda.lin_decode_step(x, x, x, g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError):
        kda.lin_bwd(x, x, x, g, x, cu)
    with pytest.raises(ValueError):
        kda.block_norm(x)
    with pytest.raises(ValueError):
        kda.block_norm_bwd(x, None, x)
