"""Linear attention with one decay a head and the query/key norm with rotation:
argument checks on the host, and the fp64 oracle against differences and the
chunk form (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_30_b200 as kda
import oracle.linear as ol
from kimi_delta_attention_30_b200.autograd import linear_chunk, norm_rope

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_SEQ, E_WS = 0, -1, -2, -3, -4, -6, -7
vp = lambda x: None if x is None else ctypes.c_void_p(x)


def _cu(cu):
    if cu is None:
        return None
    keep = (ctypes.c_int32 * len(cu))(*cu)
    return ctypes.cast(keep, ctypes.POINTER(ctypes.c_int32))


def _fwd(**kw):
    """kda_linear_chunk_fwd with fake (never dereferenced) device pointers."""
    a = dict(q=0x10000, k=0x20000, v=0x30000, la=0x40000, decay=0, dtype=1, s0=None, cu=None, n=0, B=1, T=256, H=2,
             dk=64, dv=64, o=0x60000, fs=None, ws=0x100000, wsb=1 << 40)
    a.update(kw)
    return kda.lib().kda_linear_chunk_fwd(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["la"]), a["decay"], a["dtype"],
                                          vp(a["s0"]), _cu(a["cu"]), a["n"], a["B"], a["T"], a["H"], a["dk"], a["dv"],
                                          vp(a["o"]), vp(a["fs"]), vp(a["ws"]), a["wsb"], None)


def _bwd(**kw):
    a = dict(q=0x10000, k=0x20000, v=0x30000, la=0x40000, decay=0, dtype=0, s0=None, cu=None, n=0, B=1, T=256, H=2,
             dk=128, dv=128, do=0x60000, dfs=None, dq=0x70000, dk_=0x80000, dv_=0x90000, dla=0xa0000, ds0=None,
             ws=0x100000, wsb=1 << 40)
    a.update(kw)
    return kda.lib().kda_linear_chunk_bwd(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["la"]), a["decay"], a["dtype"],
                                          vp(a["s0"]), _cu(a["cu"]), a["n"], a["B"], a["T"], a["H"], a["dk"], a["dv"],
                                          vp(a["do"]), vp(a["dfs"]), vp(a["dq"]), vp(a["dk_"]), vp(a["dv_"]),
                                          vp(a["dla"]), vp(a["ds0"]), vp(a["ws"]), a["wsb"], None)


COMMON = [
    (dict(dtype=5), E_DTYPE), (dict(decay=2), E_SHAPE), (dict(dk=96), E_SHAPE), (dict(dv=32), E_SHAPE),
    (dict(H=0), E_SHAPE), (dict(H=65536), E_SHAPE), (dict(B=-1), E_SHAPE), (dict(T=-1), E_SHAPE),
    (dict(q=None), E_NULL), (dict(la=None), E_NULL), (dict(ws=None), E_WS), (dict(wsb=16), E_WS),
    (dict(k=0x20004), E_ALIGN), (dict(la=0x40002), E_ALIGN), (dict(ws=0x100010), E_ALIGN),
    (dict(cu=[0, 100, 50, 256], n=3), E_SEQ), (dict(cu=[1, 256], n=1), E_SEQ), (dict(cu=[0, 200], n=1), E_SEQ),
    (dict(cu=[0, 256], n=1, B=2), E_SEQ), (dict(cu=[0], n=0), E_SEQ),
    (dict(T=0x7fffffff, H=1), E_SHAPE), (dict(T=1 << 30, B=4), E_SHAPE),
]


@pytest.mark.parametrize("dtype,d", [(1, 64), (0, 128)])
@pytest.mark.parametrize("kw,code", COMMON + [(dict(o=None), E_NULL), (dict(s0=0x70004), E_ALIGN)])
def test_fwd_rejects_before_launch(kw, code, dtype, d):
    assert _fwd(**{"dtype": dtype, "dk": d, "dv": d, **kw}) == code


@pytest.mark.parametrize("dtype,d", [(1, 64), (0, 128)])
@pytest.mark.parametrize("kw,code", COMMON + [
    (dict(do=None), E_NULL), (dict(dla=None), E_NULL), (dict(dq=None), E_NULL), (dict(dv_=0x90008), E_ALIGN),
    (dict(decay=1, dla=None, wsb=16), E_WS)])   # a fixed decay needs no dlog_alpha
def test_bwd_rejects_before_launch(kw, code, dtype, d):
    assert _bwd(**{"dtype": dtype, "dk": d, "dv": d, **kw}) == code


def test_decode_rejects_before_launch():
    f = kda.lib().kda_linear_decode_step
    args = [vp(0x10000)] * 4
    assert f(*args, 0, 3, vp(0x70000), 4, 2, 64, 64, vp(0x80000), None) == E_DTYPE
    assert f(*args, 2, 0, vp(0x70000), 4, 2, 64, 64, vp(0x80000), None) == E_SHAPE
    assert f(*args, 0, 0, vp(0x70000), 4, 2, 96, 64, vp(0x80000), None) == E_SHAPE
    assert f(*args, 0, 0, vp(0x70000), -1, 2, 64, 64, vp(0x80000), None) == E_SHAPE
    assert f(*args, 0, 0, None, 4, 2, 64, 64, vp(0x80000), None) == E_NULL
    assert f(*args, 0, 0, vp(0x70000), 4, 2, 64, 64, None, None) == E_NULL
    assert f(*args, 0, 0, vp(0x70004), 4, 2, 64, 64, vp(0x80000), None) == E_ALIGN
    assert f(*args, 0, 0, vp(0x70000), 0, 2, 64, 64, vp(0x80000), None) == OK   # N = 0: no work


def test_wait_limit_knows_the_linear_kernels():
    f = kda.lib().kda_set_test_wait_limit
    for bits in (8, 16, 32, 8 | 16 | 32 | 3):
        assert f(bits, 1000) == OK
    assert f(64, 1000) == E_SHAPE and f(8 | 64, 1000) == E_SHAPE and f(8, 0) == E_SHAPE
    assert f(0, 0) == OK   # disarm


def test_workspace_sizes():
    for dt, d in ((1, 64), (1, 128), (0, 64), (0, 128)):
        one = kda.linear_workspace_size(1, 1, 1, d, d, dt)
        assert 0 < one <= kda.linear_workspace_size(4, 4096, 16, d, d, dt)
        assert kda.linear_workspace_size(4, 4096, 16, d, d, dt) < kda.linear_workspace_size(4, 4096, 16, d, d, dt,
                                                                                            backward=True)
        assert kda.linear_workspace_size(1, 0, 1, d, d, dt) > 0
        assert kda.linear_workspace_size(1, 10, 1, d, d, dt, cu_seqlens=[0, 4, 4, 10]) > 0
        assert kda.linear_workspace_size(1, 10, 1, d, d, dt, cu_seqlens=[0, 6, 4, 10]) == 0
    assert kda.linear_workspace_size(1, 10, 1, 96, 64, 0) == 0
    assert kda.linear_workspace_size(1, 10, 1, 64, 64, 7) == 0


def _rows(data=0x10000, t=128, h=64):
    return kda._Rows(data, t, h)


def _rope(bwd=False, **kw):
    a = dict(q=_rows(), k=_rows(), wq=0x20000, wk=0x20000, wdt=0, pos=0x30000, fr=0x40000, dtype=0, T=8, Hq=2, Hk=2,
             d=64, rot=64, eps=1e-6, inter=0, qo=_rows(), ko=_rows(), dq=_rows(), dk=_rows(), dwq=0x50000,
             dwk=0x60000, ws=0x100000, wsb=1 << 30)
    a.update(kw)
    args = [a["q"], a["k"], vp(a["wq"]), vp(a["wk"]), a["wdt"], vp(a["pos"]), vp(a["fr"]), a["dtype"], a["T"], a["Hq"],
            a["Hk"], a["d"], a["rot"], a["eps"], a["inter"], a["qo"], a["ko"]]
    if not bwd:
        return kda.lib().kda_qk_norm_rope(*args, None)
    return kda.lib().kda_qk_norm_rope_bwd(*args, a["dq"], a["dk"], vp(a["dwq"]), vp(a["dwk"]), vp(a["ws"]), a["wsb"],
                                          None)


ROPE = [
    (dict(dtype=4), E_DTYPE), (dict(wdt=4), E_DTYPE), (dict(d=96), E_SHAPE), (dict(rot=8), E_SHAPE),
    (dict(rot=80), E_SHAPE), (dict(rot=-16), E_SHAPE), (dict(eps=-1.0), E_SHAPE), (dict(eps=float("nan")), E_SHAPE),
    (dict(Hq=0), E_SHAPE), (dict(Hk=70000), E_SHAPE), (dict(T=-1), E_SHAPE), (dict(T=1 << 31), E_SHAPE),
    (dict(q=None), E_NULL), (dict(k=_rows(0)), E_NULL), (dict(pos=None), E_NULL), (dict(fr=None), E_NULL),
    (dict(q=_rows(0x10008)), E_ALIGN), (dict(k=_rows(t=132)), E_ALIGN), (dict(q=_rows(t=-128)), E_SHAPE),
    (dict(wq=0x20004), E_ALIGN), (dict(pos=0x30002), E_ALIGN),
]


@pytest.mark.parametrize("kw,code", ROPE + [
    (dict(qo=_rows(t=64)), E_SHAPE),            # written rows overlap
    (dict(ko=_rows(h=0)), E_SHAPE), (dict(qo=_rows(t=64, h=128)), E_SHAPE),
    (dict(qo=_rows(t=192)), E_SHAPE),           # in place, but not the same rows
    (dict(qo=_rows(t=1 << 62, h=1 << 62)), E_SHAPE), (dict(ko=_rows(t=0, h=1 << 62)), E_SHAPE)])
def test_norm_rope_rejects_before_launch(kw, code):
    assert _rope(**kw) == code


@pytest.mark.parametrize("kw,code", ROPE + [
    (dict(dq=_rows(t=64)), E_SHAPE), (dict(ws=None), E_WS), (dict(wsb=8), E_WS), (dict(ws=0x100040), E_ALIGN),
    (dict(dwq=0x50004), E_ALIGN), (dict(qo=_rows(0)), E_NULL), (dict(dk=_rows(t=192)), E_SHAPE)])
def test_norm_rope_bwd_rejects_before_launch(kw, code):
    assert _rope(bwd=True, **kw) == code


def test_norm_rope_without_tokens_is_no_work():
    assert _rope(T=0) == OK
    assert _rope(bwd=True, T=0, dwq=None, dwk=None) == OK


def test_binding_refuses():
    x = torch.zeros(1, 4, 1, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_chunk_fwd(x, x, x, torch.zeros(1, 4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_chunk_bwd(x, x, x, torch.zeros(1, 4, 1), x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.linear_decode_step(x[0], x[0], x[0], torch.zeros(4, 1), torch.zeros(4, 1, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        kda.qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="dtype"):
        kda.linear_chunk_fwd(x.half(), x, x, torch.zeros(1, 4, 1))


# ---- the oracle itself -----------------------------------------------------------

def _case(seed=0, H=2, dk=5, dv=4, lens=(7, 0, 3)):
    r = np.random.default_rng(seed)
    n = sum(lens)
    ss = np.concatenate([[0], np.cumsum(lens)])
    return (r.normal(size=(n, H, dk)), r.normal(size=(n, H, dk)), r.normal(size=(n, H, dv)),
            -np.abs(r.normal(size=(n, H))), ss, r.normal(size=(len(lens), H, dk, dv)))


def test_oracle_gradients_equal_differences():
    q, k, v, la, ss, s0 = _case()
    r = np.random.default_rng(5)
    do, df = r.normal(size=v.shape), r.normal(size=s0.shape)
    g = ol.backward(q, k, v, la, ss, do, df, s0)

    def loss(q, k, v, la, s0):
        o, f = ol.forward(q, k, v, la, ss, s0)
        return (o * do).sum() + (f * df).sum()

    args = [q, k, v, la, s0]
    for i, name in enumerate(("dq", "dk", "dv", "dlog_alpha", "d_init_state")):
        u = r.normal(size=args[i].shape)
        h = 1e-5
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + h * u, args[i] - h * u
        # central differences: error h^2 times third derivatives, and 1e-16 / h of rounding
        assert abs((loss(*up) - loss(*dn)) / (2 * h) - (g[name] * u).sum()) <= 1e-7 * (1 + abs((g[name] * u)).sum())


@pytest.mark.parametrize("C", [1, 3, 4, 16])
def test_chunk_form_and_its_decay_gradient(C):
    """The kernels' chunk form, fp64: o, the carried state and the four sums of dlog_alpha."""
    q, k, v, la, _, s0 = _case(seed=2, lens=(11,))
    r = np.random.default_rng(3)
    do, df = r.normal(size=v.shape), r.normal(size=s0.shape)
    ss = np.array([0, 11])
    o_ref, f_ref = ol.forward(q, k, v, la, ss, s0)
    ref = ol.backward(q, k, v, la, ss, do, df, s0)
    for h in range(q.shape[1]):
        S, starts, o = s0[0, h], [], []
        parts = [(a, min(a + C, 11)) for a in range(0, 11, C)]
        for a, b in parts:
            g = np.cumsum(la[a:b, h])
            D = np.tril(np.exp(np.minimum(g[:, None] - g[None], 0)))
            Q, K, V = q[a:b, h], k[a:b, h], v[a:b, h]
            starts.append(S)
            o.append(np.exp(g)[:, None] * (Q @ S) + ((Q @ K.T) * D) @ V)
            S = np.exp(g[-1]) * S + (np.exp(g[-1] - g)[:, None] * K).T @ V
        np.testing.assert_allclose(np.concatenate(o), o_ref[:, h], rtol=0, atol=1e-12 * np.abs(o_ref).max() * 100)
        np.testing.assert_allclose(S, f_ref[0, h], rtol=0, atol=1e-12 * np.abs(f_ref).max() * 100)
        dS = df[0, h]
        for (a, b), S in zip(reversed(parts), reversed(starts)):
            g = np.cumsum(la[a:b, h])
            D = np.tril(np.exp(np.minimum(g[:, None] - g[None], 0)))
            Q, K, V, O = q[a:b, h], k[a:b, h], v[a:b, h], do[a:b, h]
            wq, wk = np.exp(g), np.exp(g[-1] - g)
            dA = (O @ V.T) * D
            qi, ki = wq[:, None] * (O @ S.T), wk[:, None] * (V @ dS.T)
            qa, ka = dA @ K, dA.T @ Q
            ra, rb = (Q * qi).sum(1), (K * ki).sum(1)
            x = (Q * qa).sum(1) - (K * ka).sum(1)
            suf = np.cumsum((ra + x)[::-1])[::-1]
            pre = np.cumsum(rb) - rb
            dla = suf + pre + np.exp(g[-1]) * (dS * S).sum()
            np.testing.assert_allclose(qi + qa, ref["dq"][a:b, h], atol=1e-11)
            np.testing.assert_allclose(ki + ka, ref["dk"][a:b, h], atol=1e-11)
            np.testing.assert_allclose(dla, ref["dlog_alpha"][a:b, h], atol=1e-11)
            dS = np.exp(g[-1]) * dS + (wq[:, None] * Q).T @ O
        np.testing.assert_allclose(dS, ref["d_init_state"][0, h], atol=1e-11)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rope_oracle_gradients_equal_differences(interleaved):
    r = np.random.default_rng(1)
    x, w, dy = r.normal(size=(4, 3, 8)), r.normal(size=8), r.normal(size=(4, 3, 8))
    pos, fr, eps = np.array([0, 5, -3, 100000]), np.array([1.0, 0.1]), 1e-3
    dx, dw = ol.norm_rope_backward(x, w, pos, fr, eps, interleaved, dy)
    f = lambda x, w: (ol.norm_rope(x, w, pos, fr, eps, interleaved) * dy).sum()
    u, z, h = r.normal(size=x.shape), r.normal(size=8), 1e-5
    assert abs((f(x + h * u, w) - f(x - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-6
    assert abs((f(x, w + h * z) - f(x, w - h * z)) / (2 * h) - (dw * z).sum()) < 1e-6
    # the rotation keeps each pair's length
    y = ol.norm_rope(x, None, pos, fr, eps, interleaved)
    np.testing.assert_allclose((y ** 2).sum(-1), ((x * ol._inv_rms(x, eps)) ** 2).sum(-1))


# ---- gradient routing ------------------------------------------------------------

def test_linear_chunk_routes_gradients():
    mk = lambda *s: torch.randn(*s).requires_grad_()
    q, k, v, la, s0 = mk(1, 6, 2, 4), mk(1, 6, 2, 4), mk(1, 6, 2, 3), mk(1, 6, 2), mk(1, 2, 4, 3)
    seen = {}

    def fwd(q, k, v, la, init_state=None, cu_seqlens=None):
        return torch.ones(1, 6, 2, 3), torch.ones(1, 2, 4, 3)

    def bwd(q, k, v, la, d_o, init_state=None, d_final_state=None, cu_seqlens=None, need_d_init_state=True):
        seen.update(d_o=d_o, df=d_final_state, cu=cu_seqlens, need=need_d_init_state)
        return (torch.full_like(q, 1.), torch.full_like(k, 2.), torch.full_like(v, 3.),
                torch.full_like(la, 4.) if la.dim() == 3 else None, torch.full((1, 2, 4, 3), 5.))

    o, fs = linear_chunk(q, k, v, la, s0, [0, 6], ops=(fwd, bwd))
    (2 * o.sum() + 3 * fs.sum()).backward()
    assert [float(t.grad.flatten()[0]) for t in (q, k, v, la, s0)] == [1, 2, 3, 4, 5]
    assert float(seen["d_o"].mean()) == 2 and float(seen["df"].mean()) == 3 and seen["cu"] == [0, 6] and seen["need"]
    fixed = torch.zeros(2).requires_grad_()
    with pytest.raises(ValueError, match="fixed decay"):
        linear_chunk(q, k, v, fixed, ops=(fwd, bwd))[0].sum().backward()


def test_norm_rope_routes_gradients():
    mk = lambda *s: torch.randn(*s).requires_grad_()
    q, k, w = mk(6, 2, 4), mk(6, 1, 4), mk(4)
    fwd = lambda q, k, *a, **kw: (q * 1, k * 1)
    bwd = lambda q, k, *a, **kw: (torch.full_like(q, 1.), torch.full_like(k, 2.), torch.full((4,), 3.), None)
    y, z = norm_rope(q, k, w, None, torch.arange(6), torch.ones(2), ops=(fwd, bwd))
    (y.sum() + z.sum()).backward()
    assert [float(t.grad.flatten()[0]) for t in (q, k, w)] == [1, 2, 3]


def test_gradients_of_gradients_are_refused():
    """The backward kernels are not differentiable: a penalty on a gradient would otherwise lose
    what flows through the operator without a word."""
    from kimi_delta_attention_30_b200.autograd import kda_chunk
    mk = lambda *s: torch.randn(*s).requires_grad_()
    q, k, v, la = mk(1, 6, 2, 4), mk(1, 6, 2, 4), mk(1, 6, 2, 4), mk(1, 6, 2)
    state = torch.ones(1, 2, 4, 4)
    lin = (lambda q, k, v, la, **kw: (v * 1, state),
           lambda q, k, v, la, d_o, **kw: (q * d_o, k * d_o, v * d_o, la * 1, None))
    kda3 = (lambda q, k, v, la, b, **kw: (v * 1, state),
            lambda q, k, v, la, b, d_o, **kw: (q * d_o, k * d_o, v * d_o, la * 1, b * 1, None))
    rope = (lambda q, k, *a, **kw: (q * 1, k * 1), lambda q, k, w, x, p, f, dq, dk, **kw: (q * dq, k * dk, None, None))
    for out in (linear_chunk(q, k, v, la, ops=lin)[0], kda_chunk(q, k, v, q.clone(), la, ops=kda3)[0],
                norm_rope(q, k, None, None, torch.arange(6), torch.ones(2), ops=rope)[0]):
        (g,) = torch.autograd.grad(out.square().sum(), [q], create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.square().sum() + out.sum()).backward()


@pytest.mark.parametrize("make", [list, np.array, torch.tensor], ids=["list", "numpy", "torch"])
def test_offsets_of_the_forward_call_are_those_of_the_backward(make):
    """A caller that fills one buffer with every batch's offsets."""
    from kimi_delta_attention_30_b200.autograd import kda_chunk
    mk = lambda *s: torch.randn(*s).requires_grad_()
    q, v, la = mk(1, 6, 2, 4), mk(1, 6, 2, 4), mk(1, 6, 2)
    seen = []
    fwd = lambda *a, cu_seqlens=None, **kw: (seen.append(list(cu_seqlens)), (a[2] * 1, torch.ones(2, 2, 4, 4)))[1]
    bwd = lambda *a, cu_seqlens=None, **kw: (seen.append(list(cu_seqlens)), (*a[:-1], None))[1]
    for f, args in ((linear_chunk, (q, q, v, la)), (kda_chunk, (q, q, v, q, la))):
        cu = make([0, 2, 6])
        seen.clear()
        o, _ = f(*args, cu_seqlens=cu, ops=(fwd, bwd))
        cu[1] = 5
        o.sum().backward()
        assert seen == [[0, 2, 6]] * 2 and all(type(x) is int for x in seen[0])


# ---- results in an input's memory --------------------------------------------------

_MB = 1 << 20


def _apart():
    """Arguments whose arrays lie apart (1 MB each)."""
    names = ("q", "k", "v", "la", "s0", "o", "fs", "do", "dfs", "dq", "dk_", "dv_", "dla", "ds0", "ws")
    return {n: (i + 1) * _MB for i, n in enumerate(names)}


FWD = ("q", "k", "v", "la", "s0", "o", "fs", "ws")
BWD = ("q", "k", "v", "la", "s0", "do", "dfs", "dq", "dk_", "dv_", "dla", "ds0", "ws")


@pytest.mark.parametrize("dtype,d", [(1, 64), (0, 128)])
def test_results_that_overlap_inputs_are_refused(dtype, d):
    if torch.cuda.is_available():
        pytest.skip("valid arguments would launch")
    size = dict(dtype=dtype, dk=d, dv=d, T=256, H=2)
    far = _apart()
    fwd = {n: far[n] for n in FWD}
    bwd = {n: far[n] for n in BWD}
    ok = _fwd(**size, **fwd)
    assert ok not in (OK, E_SHAPE, E_ALIGN, E_NULL, E_WS)          # accepted but for the missing device
    assert _bwd(**size, **bwd) == ok
    nbytes = 256 * 2 * d * (4 if dtype else 2)
    for r in ("o", "fs"):
        for x in ("q", "k", "v", "la", "s0"):
            for shift in (0, 16):                                   # the same start, and partly
                want = ok if (r, x, shift) == ("fs", "s0", 0) else E_SHAPE
                assert _fwd(**size, **{**fwd, r: fwd[x] + shift}) == want, (r, x)
    assert _fwd(**size, **{**fwd, "o": fwd["v"] - nbytes}) == ok    # one behind the other
    assert _fwd(**size, **{**fwd, "o": fwd["v"] - nbytes + 16}) == E_SHAPE
    for r in ("dq", "dk_", "dv_", "dla", "ds0"):
        for x in ("q", "k", "v", "la", "do", "s0", "dfs"):
            for shift in (0, 16):
                want = ok if (r, x, shift) == ("ds0", "dfs", 0) else E_SHAPE
                assert _bwd(**size, **{**bwd, r: bwd[x] + shift}) == want, (r, x)
    assert _bwd(**size, **{**bwd, "decay": 1, "dla": bwd["q"]}) == ok   # not written
    f = kda.lib().kda_linear_decode_step

    def dec(**kw):
        a = {n: far[n] for n in ("q", "k", "v", "la", "s0", "o")}
        a.update(kw)
        return f(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["la"]), 0, dtype, vp(a["s0"]), 5, 2, d, d, vp(a["o"]), None)

    assert dec() == ok
    for r, x in [("o", x) for x in ("q", "k", "v", "la", "s0")] + [("s0", x) for x in ("q", "k", "v", "la")]:
        assert dec(**{r: far[x]}) == E_SHAPE and dec(**{r: far[x] + 16}) == E_SHAPE, (r, x)


def test_decays_need_four_bytes():
    if torch.cuda.is_available():
        pytest.skip("valid arguments would launch")
    far = _apart()
    for dtype, d in ((1, 64), (0, 128)):
        size = dict(dtype=dtype, dk=d, dv=d, T=256, H=2)
        fwd, bwd = ({n: far[n] for n in names} for names in (FWD, BWD))
        ok = _fwd(**size, **fwd)
        for off in (4, 8, 12):
            assert _fwd(**size, **{**fwd, "la": far["la"] + off}) == ok
            assert _fwd(**size, **{**fwd, "la": far["la"] + off, "decay": 1}) == ok
            assert _bwd(**size, **{**bwd, "la": far["la"] + off, "dla": far["dla"] + off}) == ok
        assert _fwd(**size, **{**fwd, "la": far["la"] + 2}) == E_ALIGN
        assert _bwd(**size, **{**bwd, "dla": far["dla"] + 2}) == E_ALIGN


@pytest.mark.parametrize("dtype,d", [(1, 64), (0, 128)])
def test_more_sequence_heads_than_a_grid_takes_are_refused(dtype, d):
    """Empty sequences take no memory, so their number is bounded by the launch alone."""
    n = 20000
    kw = dict(dtype=dtype, dk=d, dv=d, T=1, H=65535, cu=[0] * n + [1], n=n)
    assert _fwd(**kw) == E_SHAPE and _bwd(**kw) == E_SHAPE


def test_arrays_without_elements_overlap_nothing():
    if torch.cuda.is_available():
        pytest.skip("valid arguments would launch")
    far = _apart()
    for dtype, d in ((1, 64), (0, 128)):
        fwd = {n: far[n] for n in FWD}
        size = dict(dtype=dtype, dk=d, dv=d, H=2)
        ok = _fwd(**size, T=256, **fwd)
        assert _fwd(**size, T=0, **{**fwd, "o": fwd["s0"] + 256}) == ok
        assert _fwd(**size, T=0, **{**fwd, "fs": fwd["s0"] + 256}) == E_SHAPE
