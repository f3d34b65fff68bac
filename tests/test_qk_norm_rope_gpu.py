"""The query/key norm with rotation on the GPU against fp64.

Tolerances.  fp32: the norm's sum of 128 squares (2^-17 at most, halved by the root),
the root (2^-22), three products, the rotation's two products and a sum, its cosines
and sines (2^-21 absolute, with the angle's remainder rounded to fp32: pi 2^-23); an
output is off by at most 2^-16 (|y_a| + |y_b|) of its pair.  Gradients: the same with
two more sums of 128 terms, 2^-15 of the terms' magnitudes; weight gradients sum n rows
in fp32 through a tree at most 700 additions deep: 2^-14 of the magnitudes.  bf16
results: 2^-8 of the value besides.
"""
import numpy as np
import pytest
import torch

import oracle.linear as ol
from kda_inputs import to_f64

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def make(dt, lead, Hq, Hk, d, rot, wdt, fused, far=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = int(np.prod(lead))
    r = lambda *s: torch.randn(*s, generator=g)
    if fused:
        x = r(*lead, Hq + 2 * Hk, d).to(DT[dt]).cuda()
        q, k = x[..., :Hq, :], x[..., Hq:Hq + Hk, :]
    else:
        q, k = r(*lead, Hq, d).to(DT[dt]).cuda(), r(*lead, Hk, d).to(DT[dt]).cuda()
    w = [None if wdt is None else (1 + 0.2 * r(d)).to(DT[wdt]).cuda() for _ in range(2)]
    hi = 2 ** 31 - 1 if far else 4000
    pos = torch.randint(-hi - 1 if far else 0, hi, (n,), generator=g).to(torch.int32).reshape(lead).cuda()
    fr = (10000.0 ** (-torch.arange(0, max(rot, 2), 2) / max(rot, 2))).float().cuda()[:rot // 2]
    dy = [r(*lead, H, d).to(DT[dt]).cuda() for H in (Hq, Hk)]
    return dict(q=q, k=k, wq=w[0], wk=w[1], pos=pos if rot else None, fr=fr if rot else None, dq=dy[0], dk=dy[1])


def flat(t):
    return to_f64(t).reshape(-1, *t.shape[-2:])


def turns(x):
    return (np.zeros(flat(x["q"]).shape[0]), np.zeros(0)) if x["fr"] is None else (to_f64(x["pos"]).reshape(-1),
                                                                                   to_f64(x["fr"]))


def pair_mag(y, rot, interleaved):
    """|y_a| + |y_b| of every channel's pair."""
    m = np.abs(y)
    out = np.array(m)
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    out[..., a] = out[..., b] = m[..., a] + m[..., b]
    return out


def close(label, got, ref, bound):
    got = to_f64(got).reshape(ref.shape)
    assert np.isfinite(got).all(), label
    worst = float((np.abs(got - ref) / np.maximum(bound, 1e-30)).max())
    assert worst <= 1.0, f"{label}: {worst:.3f} of the bound"


CASES = [  # dtype, tokens, Hq, Hk, d, rot, weights, fused view, far positions, neighbours
    ("bf16", (1,), 1, 1, 128, 128, "bf16", False, False, False),
    ("bf16", (2, 37), 4, 2, 128, 128, "bf16", True, False, False),
    ("bf16", (5,), 3, 1, 64, 64, "f32", True, True, True),
    ("f32", (3, 11), 6, 2, 64, 32, "f32", False, False, True),
    ("f32", (70,), 5, 5, 128, 64, None, True, True, False),
    ("bf16", (33,), 2, 7, 128, 32, None, False, False, False),
    ("f32", (9,), 1, 3, 64, 16, "bf16", False, False, False),
    ("bf16", (4, 3, 5), 2, 2, 64, 0, "bf16", True, False, False),
    ("bf16", (3000,), 17, 3, 128, 128, "f32", True, False, False),
]
IDS = ["-".join(str(y) for y in c).replace(" ", "") for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(cuda_ok, case):
    import kimi_delta_attention_30_b200 as kda
    dt, lead, Hq, Hk, d, rot, wdt, fused, far, inter = case
    x = make(dt, lead, Hq, Hk, d, rot, wdt, fused, far, seed=1)
    q, k = kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["fr"], eps=EPS, interleaved=inter)
    torch.cuda.synchronize()
    pos, fr = turns(x)
    for name, got, src, w in (("q", q, x["q"], x["wq"]), ("k", k, x["k"], x["wk"])):
        assert got.shape == src.shape and got.dtype == src.dtype and got.is_contiguous()
        w = None if w is None else to_f64(w)
        ref = ol.norm_rope(flat(src), w, pos, fr, EPS, inter)
        y = flat(src) * ol._inv_rms(flat(src), EPS) * (1.0 if w is None else w)
        close(name, got, ref, 2.0 ** -16 * pair_mag(y, rot, inter) + (2.0 ** -8 * np.abs(ref) if dt == "bf16" else 0))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(cuda_ok, case):
    import kimi_delta_attention_30_b200 as kda
    dt, lead, Hq, Hk, d, rot, wdt, fused, far, inter = case
    x = make(dt, lead, Hq, Hk, d, rot, wdt, fused, far, seed=2)
    got = kda.qk_norm_rope_bwd(x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["fr"], x["dq"], x["dk"], eps=EPS,
                               interleaved=inter)
    again = kda.qk_norm_rope_bwd(x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["fr"], x["dq"], x["dk"], eps=EPS,
                                 interleaved=inter)
    torch.cuda.synchronize()
    assert all(a is b or torch.equal(a, b) for a, b in zip(got, again))
    pos, fr = turns(x)
    for i, (src, w, dy) in enumerate(((x["q"], x["wq"], x["dq"]), (x["k"], x["wk"], x["dk"]))):
        w64 = None if w is None else to_f64(w)
        t, g = flat(src), flat(dy)
        dx, dw = ol.norm_rope_backward(t, w64, pos, fr, EPS, inter, g)
        gm = pair_mag(g, rot, inter)                     # magnitudes after turning back
        r = ol._inv_rms(t, EPS)
        hm = gm if w64 is None else gm * np.abs(w64)
        mag = r * hm + np.abs(t) * r ** 3 * (hm * np.abs(t)).mean(-1, keepdims=True)
        close(f"dx{i}", got[i], dx, 2.0 ** -15 * mag + (2.0 ** -8 * np.abs(dx) if dt == "bf16" else 0))
        if w is None:
            assert got[2 + i] is None
        else:
            assert got[2 + i].dtype == w.dtype
            close(f"dw{i}", got[2 + i], dw, 2.0 ** -14 * (gm * np.abs(t) * r).sum((0, 1)) +
                  (2.0 ** -8 * np.abs(dw) if wdt == "bf16" else 0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_in_place_and_given_outputs(cuda_ok, dt):
    import kimi_delta_attention_30_b200 as kda
    x = make(dt, (300,), 8, 4, 128, 128, dt, True, seed=3)
    args = (x["wq"], x["wk"], x["pos"], x["fr"])
    want = kda.qk_norm_rope(x["q"], x["k"], *args)
    rest = x["q"]._base[..., 12:, :].clone()
    wide = torch.full((300, 10, 128), 3.0, dtype=DT[dt], device="cuda")     # outputs with gaps
    got = kda.qk_norm_rope(x["q"], x["k"], *args, q_out=wide[:, :8], k_out=torch.empty_like(want[1]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and (wide[:, 8:] == 3.0).all()
    heads_first = torch.empty(8, 300, 128, dtype=DT[dt], device="cuda").transpose(0, 1)
    got = kda.qk_norm_rope(x["q"], x["k"], *args, q_out=heads_first)
    assert torch.equal(got[0], want[0])
    q, k = kda.qk_norm_rope(x["q"], x["k"], *args, q_out=x["q"], k_out=x["k"])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x["q"]._base[..., 12:, :], rest)
    # gradients in place of their upstream gradients
    y = make(dt, (300,), 8, 4, 128, 128, dt, True, seed=4)
    a = (y["q"], y["k"], y["wq"], y["wk"], y["pos"], y["fr"])
    want = kda.qk_norm_rope_bwd(*a, y["dq"], y["dk"])
    got = kda.qk_norm_rope_bwd(*a, y["dq"], y["dk"], grads=(y["dq"], y["dk"], None, want[3].clone()))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[3], want[3])


def test_zero_rows_and_refusals(cuda_ok):
    import kimi_delta_attention_30_b200 as kda
    x = make("bf16", (4,), 2, 2, 64, 64, "bf16", False, seed=5)
    x["q"].zero_()
    q, _ = kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["fr"], eps=0.0)
    assert not q.any()
    g = kda.qk_norm_rope_bwd(x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["fr"], x["dq"], x["dk"], eps=0.0)
    assert not g[0].any() and not g[2].any()
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    q, k = kda.qk_norm_rope(e, e, x["wq"], x["wk"], x["pos"][:0], x["fr"])
    assert q.shape == e.shape
    g = kda.qk_norm_rope_bwd(e, e, x["wq"], x["wk"], x["pos"][:0], x["fr"], e, e)
    assert not g[2].any() and not g[3].any()
    bad = x["k"].transpose(1, 2).contiguous().transpose(1, 2)          # last dimension not contiguous
    for kw, text in ((dict(k=bad), "contiguous"), (dict(positions=x["pos"].long()), "dtype"),
                     (dict(positions=x["pos"][:3]), "shape"), (dict(positions=None), "positions"),
                     (dict(q_weight=x["wq"][:32]), "shape"), (dict(inv_freq=x["fr"].cpu()), "CUDA")):
        a = dict(q=x["q"], k=x["k"], q_weight=x["wq"], k_weight=x["wk"], positions=x["pos"], inv_freq=x["fr"])
        with pytest.raises(ValueError, match=text):
            kda.qk_norm_rope(**{**a, **kw})
    with pytest.raises(kda.KdaError):                                   # overlapping written rows
        kda.qk_norm_rope(x["q"], x["k"], q_out=x["q"][:1].expand(4, 2, 64))


def test_streams_graph_and_autograd(cuda_ok):
    import kimi_delta_attention_30_b200 as kda
    from kimi_delta_attention_30_b200.autograd import norm_rope
    x = make("bf16", (200,), 8, 2, 128, 64, "bf16", True, seed=6)
    a = (x["q"], x["k"], x["wq"], x["wk"], x["pos"], x["fr"])
    want = kda.qk_norm_rope(*a) + kda.qk_norm_rope_bwd(*a, x["dq"], x["dk"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = kda.qk_norm_rope(*a, stream=s) + kda.qk_norm_rope_bwd(*a, x["dq"], x["dk"], stream=s)
    s.synchronize()
    assert all(torch.equal(t, u) for t, u in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kda.qk_norm_rope(*a) + kda.qk_norm_rope_bwd(*a, x["dq"], x["dk"])
    for t in out:
        t.fill_(9.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(t, u) for t, u in zip(want, out))
    leaves = [t.clone().requires_grad_() for t in a[:4]]
    q, k = norm_rope(*leaves, x["pos"], x["fr"])
    torch.autograd.backward([q, k], [x["dq"], x["dk"]])
    assert all(torch.equal(t.grad, u) for t, u in zip(leaves, want[2:]))


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dt,d,rot", [("bf16", 128, 64), ("f32", 64, 64), ("f32", 128, 0)])
def test_nan_reaches_its_row_and_no_other(cuda_ok, dt, d, rot, inter):
    """The norm divides a whole row by one number, so a NaN channel is a NaN row."""
    import kimi_delta_attention_30_b200 as kda
    x = make(dt, (9,), 6, 2, d, rot, dt, False, seed=11)
    args = (x["wq"], x["wk"], x["pos"], x["fr"])
    kw = dict(eps=EPS, interleaved=inter)
    want = kda.qk_norm_rope(x["q"], x["k"], *args, **kw)
    grads = kda.qk_norm_rope_bwd(x["q"], x["k"], *args, x["dq"], x["dk"], **kw)
    q = x["q"].clone()
    q[3, 4, d - 1] = q[7, 0, 0] = float("nan")
    bad = torch.zeros(9, 6, dtype=torch.bool, device="cuda")
    bad[3, 4] = bad[7, 0] = True
    for eps in (EPS, 0.0):
        got, k = kda.qk_norm_rope(q, x["k"], *args, eps=eps, interleaved=inter)
        assert got[bad].isnan().all() and got[~bad].isfinite().all()
        if eps == EPS:
            assert torch.equal(got[~bad], want[0][~bad]) and torch.equal(k, want[1])
    g = kda.qk_norm_rope_bwd(q, x["k"], *args, x["dq"], x["dk"], **kw)
    assert g[0][bad].isnan().all() and torch.equal(g[0][~bad], grads[0][~bad]) and torch.equal(g[1], grads[1])
    assert g[2].isnan().all() and torch.equal(g[3], grads[3])
    # an upstream gradient's NaN: its row of dx through the mean, and the weight channels of its pair
    dq = x["dq"].clone()
    dq[2, 1, 5] = float("nan")
    g = kda.qk_norm_rope_bwd(x["q"], x["k"], *args, dq, x["dk"], **kw)
    bad[:] = False
    bad[2, 1] = True
    assert g[0][bad].isnan().all() and torch.equal(g[0][~bad], grads[0][~bad])
    pair = [5] if rot == 0 else [4, 5] if inter else [5, 5 + rot // 2]
    one = torch.zeros(d, dtype=torch.bool, device="cuda")
    one[pair] = True
    assert g[2][one].isnan().all() and torch.equal(g[2][~one], grads[2][~one])


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("dt,d,rot", [("bf16", 128, 32), ("f32", 64, 16), ("f32", 128, 0)])
def test_channels_that_do_not_turn_stay_apart(cuda_ok, dt, d, rot, inter):
    """An infinite channel behind the rotated ones: its row's scale is 0, so it is NaN and every other
    channel 0; an infinite upstream gradient there reaches one weight channel."""
    import kimi_delta_attention_30_b200 as kda
    x = make(dt, (5,), 3, 1, d, rot, dt, False, seed=12)
    args = (x["wq"], x["wk"], x["pos"], x["fr"])
    for c in (rot, rot + 9, d - 1):
        q = x["q"].clone()
        q[1, 2, c] = float("inf")
        got, _ = kda.qk_norm_rope(q, x["k"], *args, eps=EPS, interleaved=inter)
        row = got[1, 2]
        assert row[c].isnan() and not row[:c].any() and not row[c + 1:].any()
        dq = x["dq"].clone()
        want = kda.qk_norm_rope_bwd(x["q"], x["k"], *args, dq, x["dk"], eps=EPS, interleaved=inter)
        dq[1, 2, c] = float("inf")
        g = kda.qk_norm_rope_bwd(x["q"], x["k"], *args, dq, x["dk"], eps=EPS, interleaved=inter)
        one = torch.zeros(d, dtype=torch.bool, device="cuda")
        one[c] = True
        assert not g[2][one].isfinite().any() and torch.equal(g[2][~one], want[2][~one])


def test_positions_without_frequencies_are_refused(cuda_ok):
    """Either both or neither: the norm alone is no answer to a call with positions."""
    import kimi_delta_attention_30_b200 as kda
    x = make("bf16", (4,), 2, 2, 64, 64, "bf16", False, seed=13)
    with pytest.raises(ValueError, match="inv_freq is required"):
        kda.qk_norm_rope(x["q"], x["k"], x["wq"], x["wk"], x["pos"])
    with pytest.raises(ValueError, match="inv_freq is required"):
        kda.qk_norm_rope_bwd(x["q"], x["k"], x["wq"], x["wk"], x["pos"], None, x["dq"], x["dk"])


FEW_HEADS = [   # many tokens, fewer heads a side than a warp takes at a time
    ("bf16", (20011,), 1, 1, 128, 128, "bf16", True, False, False),
    ("bf16", (3, 5003), 4, 1, 64, 32, "f32", False, True, True),
    ("f32", (9001,), 2, 1, 128, 64, "f32", False, False, True),
    ("f32", (12001,), 1, 3, 64, 64, None, True, True, False),
]


@pytest.mark.parametrize("case", FEW_HEADS, ids=["-".join(str(y) for y in c).replace(" ", "") for c in FEW_HEADS])
def test_few_heads_many_tokens(cuda_ok, case):
    test_forward(cuda_ok, case)
    test_backward(cuda_ok, case)
