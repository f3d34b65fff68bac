"""Workloads of the linear-attention operators and of the query/key norm with
rotation: the cases that are measured, their inputs, their plain forms and
their values in 64 bits.

Operators (S is a d_k x d_v state for each sequence and head, a_t = exp(log_alpha_t)
one number for each token and head, or one for each head):

* ``lin_fwd``: S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t over whole sequences
* ``lin_bwd``: gradients of sum(d_o * o) + sum(d_final_state * final_state)
* ``lin_decode``: one token of the same recurrence, the state updated in place
* ``norm_rope``: RMS norm of every query and key head, then the rotation by position
* ``norm_rope_bwd``: its gradients (inputs and norm weights)
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ---------------------------------------------------------------------

def listed():
    return [
        # a training or prompt batch of equal sequences
        dict(name="fwd_b4_h16_t4096", op="lin_fwd", dtype="bf16", B=4, T=4096, H=16, dk=128, dv=128,
             packed=False, decay="token", init=True),
        # one long prompt, fixed decay for each head
        dict(name="fwd_long_t65536_h32", op="lin_fwd", dtype="bf16", B=1, T=65536, H=32, dk=128, dv=128,
             packed=False, decay="head", init=False),
        # a serving step's prompts: 24 ragged sequences packed one after another, states carried in
        dict(name="fwd_packed24_h8", op="lin_fwd", dtype="bf16", B=24, T=1500, H=8, dk=128, dv=128,
             packed=True, decay="token", init=True),
        # the small fp32 problem, where the launches' latency counts
        dict(name="fwd_tiny_f32", op="lin_fwd", dtype="f32", B=1, T=256, H=2, dk=64, dv=64,
             packed=False, decay="token", init=False),
        # the training step that belongs to the first case
        dict(name="bwd_b4_h16_t4096", op="lin_bwd", dtype="bf16", B=4, T=4096, H=16, dk=128, dv=128,
             packed=False, decay="token", init=True),
        # fp32 training on a few ragged documents, key and value widths that differ
        dict(name="bwd_packed5_f32", op="lin_bwd", dtype="f32", B=5, T=333, H=3, dk=64, dv=128,
             packed=True, decay="token", init=True),
        # a full serving batch, one token each
        dict(name="decode_n256_h32", op="lin_decode", dtype="bf16", B=256, H=32, dk=128, dv=128,
             decay="token"),
        # a single user's token
        dict(name="decode_n1_h32", op="lin_decode", dtype="bf16", B=1, H=32, dk=128, dv=128,
             decay="head"),
        # queries and keys of a training or prompt batch, views of one fused projection
        dict(name="rope_b4_t4096_h16", op="norm_rope", dtype="bf16", B=4, T=4096, Hq=16, Hk=16, d=128,
             rot=128, interleaved=False, wdtype="bf16", fused=True, far=False),
        # one token each of a serving batch, positions far into their sequences
        dict(name="rope_decode_n256_h32", op="norm_rope", dtype="bf16", B=256, T=1, Hq=32, Hk=32, d=128,
             rot=128, interleaved=False, wdtype="bf16", fused=True, far=True),
        # the first rotation case's backward pass
        dict(name="rope_bwd_b4_t4096_h16", op="norm_rope_bwd", dtype="bf16", B=4, T=4096, Hq=16, Hk=16, d=128,
             rot=128, interleaved=False, wdtype="bf16", fused=True, far=False),
        # fp32, few key heads, half of each head rotated, neighbouring pairs
        dict(name="rope_bwd_f32_t1001", op="norm_rope_bwd", dtype="f32", B=1, T=1001, Hq=6, Hk=2, d=64,
             rot=32, interleaved=True, wdtype="f32", fused=False, far=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_bwd", "lin_decode", "norm_rope", "norm_rope_bwd"])
    if op in ("lin_fwd", "lin_bwd"):
        f32 = rng.random() < 0.25
        wide = not f32 and rng.random() < 0.8
        B, H = _log_int(rng, 1, 32), _log_int(rng, 1, 32)
        most = 2 ** 17 if f32 else 2 ** 20 if op == "lin_fwd" else 2 ** 18     # token-heads
        T = _log_int(rng, 1, max(1, min(65536 if op == "lin_fwd" else 16384, most // (B * H))))
        return dict(op=op, dtype="f32" if f32 else "bf16", B=B, T=T, H=H,
                    dk=128 if wide else rng.choice([64, 128]), dv=128 if wide else rng.choice([64, 128]),
                    packed=rng.random() < 0.5,
                    decay="token" if op == "lin_bwd" else rng.choice(["token", "head"]),
                    init=rng.random() < 0.5)
    if op == "lin_decode":
        return dict(op=op, dtype="f32" if rng.random() < 0.25 else "bf16", B=_log_int(rng, 1, 300),
                    H=_log_int(rng, 1, 32), dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    decay=rng.choice(["token", "head"]))
    d = rng.choice([64, 128])
    Hk = _log_int(rng, 1, 16)
    Hq = Hk * rng.choice([1, 1, 2, 4])
    B = _log_int(rng, 1, 16)
    f32 = rng.random() < 0.25
    T = _log_int(rng, 1, max(1, 2 ** (26 if f32 else 27) // (B * (Hq + Hk) * d)))
    return dict(op=op, dtype="f32" if f32 else "bf16", B=B, T=T, Hq=Hq, Hk=Hk, d=d,
                rot=rng.choice([d, d, d // 2, d // 4]), interleaved=rng.random() < 0.4,
                wdtype="f32" if f32 or rng.random() < 0.3 else "bf16", fused=rng.random() < 0.5,
                far=rng.random() < 0.3)


# ---- inputs --------------------------------------------------------------------

def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + salt) % (1 << 62))
    return g


def _normal(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _unit(shape, g, dtype):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dtype)


def _log_alpha(shape, g, dtype):
    """Log decays of three kinds of heads: memories of thousands, tens and single tokens."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)
    kind = torch.arange(shape[-1], device="cuda") % 3
    mid = -torch.nn.functional.softplus(x - 3.0)
    short = -torch.nn.functional.softplus(x + 1.0)
    return torch.where(kind == 0, mid, torch.where(kind == 1, -1e-3 * u, short)).to(dtype)


def _head_decay(H):
    """Fixed log decays, a geometric ladder over the heads."""
    return -torch.pow(2.0, -8.0 * (torch.arange(H, device="cuda", dtype=torch.float32) + 1.0) / H)


def _lengths(case):
    """Ragged lengths of the packed sequences: from none to T each, one of T; they belong to the case."""
    g = torch.Generator().manual_seed(case["B"] * 7919 + case["T"])
    n = torch.randint(0, case["T"] + 1, (case["B"],), generator=g).tolist()
    n[len(n) // 2] = case["T"]
    return n


def _cu(lengths):
    return [0] + torch.tensor(lengths, dtype=torch.int64).cumsum(0).tolist()


def prepare(case, seed):
    op, dt = case["op"], _DTYPE[case["dtype"]]
    st = dict(case=dict(case))
    if op in ("lin_fwd", "lin_bwd"):
        B, T, H, dk, dv = (case[x] for x in ("B", "T", "H", "dk", "dv"))
        if case["packed"]:
            st["cu"] = _cu(_lengths(case))
            rows = (1, st["cu"][-1])
        else:
            st["cu"] = None
            rows = (B, T)
        st["q"] = _unit(rows + (H, dk), _gen(seed, 1), dt)
        st["k"] = _unit(rows + (H, dk), _gen(seed, 2), dt)
        st["v"] = _normal(rows + (H, dv), _gen(seed, 3), dt)
        st["log_alpha"] = _log_alpha(rows + (H,), _gen(seed, 4), dt) if case["decay"] == "token" else _head_decay(H)
        st["init"] = 0.02 * _normal((B, H, dk, dv), _gen(seed, 5)) if case["init"] else None
        if op == "lin_bwd":
            st["d_o"] = _normal(rows + (H, dv), _gen(seed, 6), dt)
            st["d_final"] = 0.1 * _normal((B, H, dk, dv), _gen(seed, 7))
    elif op == "lin_decode":
        N, H, dk, dv = (case[x] for x in ("B", "H", "dk", "dv"))
        st["q"] = _unit((N, H, dk), _gen(seed, 1), dt)
        st["k"] = _unit((N, H, dk), _gen(seed, 2), dt)
        st["v"] = _normal((N, H, dv), _gen(seed, 3), dt)
        st["log_alpha"] = _log_alpha((N, H), _gen(seed, 4), dt) if case["decay"] == "token" else _head_decay(H)
        st["state"] = 0.02 * _normal((N, H, dk, dv), _gen(seed, 5))
    else:
        B, T, Hq, Hk, d = (case[x] for x in ("B", "T", "Hq", "Hk", "d"))
        if case["fused"]:      # views of one projection's output, the values' heads behind them
            x = _normal((B * T, (Hq + 2 * Hk) * d), _gen(seed, 1), dt)
            st["q"] = x[:, :Hq * d].unflatten(1, (Hq, d))
            st["k"] = x[:, Hq * d:(Hq + Hk) * d].unflatten(1, (Hk, d))
        else:
            st["q"] = _normal((B * T, Hq, d), _gen(seed, 1), dt)
            st["k"] = _normal((B * T, Hk, d), _gen(seed, 2), dt)
        wdt = _DTYPE[case["wdtype"]]
        st["wq"] = (1.0 + 0.1 * _normal((d,), _gen(seed, 3))).to(wdt)
        st["wk"] = (1.0 + 0.1 * _normal((d,), _gen(seed, 4))).to(wdt)
        base = torch.randint(0, 1_000_000 if case["far"] else 1024, (B, 1), generator=_gen(seed, 5), device="cuda")
        st["positions"] = (base + torch.arange(T, device="cuda")).reshape(-1).to(torch.int32)
        st["inv_freq"] = (1.0 / THETA ** (torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
                          ).to(torch.float32).cuda()
        if op == "norm_rope_bwd":
            st["d_q"] = _normal((B * T, Hq, d), _gen(seed, 6), dt)
            st["d_k"] = _normal((B * T, Hk, d), _gen(seed, 7), dt)
    return st


# ---- plain forms ---------------------------------------------------------------

CHUNK = 128


def _slots(cu, B, T, device):
    """Where each packed token sits in a [sequences, longest] grid."""
    c = torch.tensor(cu, device=device)
    n = c[1:] - c[:-1]
    longest = max(b - a for a, b in zip(cu[:-1], cu[1:]))
    seq = torch.repeat_interleave(torch.arange(len(cu) - 1, device=device), n, output_size=cu[-1])
    return seq * longest + torch.arange(cu[-1], device=device) - c[seq], longest


def _grid(x, at, n_seqs, longest):
    """Packed rows [1, T, ...] laid out as [sequences, longest, ...], zero behind each end."""
    return x.new_zeros((n_seqs * longest,) + x.shape[2:]).index_copy(0, at, x[0]).unflatten(0, (n_seqs, longest))


def _chunk_form(q, k, v, la, init):
    """The recurrence in chunks, fp32 with the decays' sums in fp64; [B, T, H, d], la [B, T, H] fp64."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n = -(-T // CHUNK)
    pad = n * CHUNK - T

    def split(x):
        x = torch.nn.functional.pad(x, (0, 0) * (x.dim() - 2) + (0, pad))
        return x.unflatten(1, (n, CHUNK)).movedim(3, 1)            # [B, H, n, C, ...]

    q, k, v, la = split(q), split(k), split(v), split(la)
    g = la.cumsum(-1)                                               # [B, H, n, C]
    later = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).triu(1)
    decay = (g[..., :, None] - g[..., None, :]).masked_fill(later, -math.inf).exp().float()
    o = ((q @ k.transpose(-1, -2)) * decay) @ v
    add = (k * (g[..., -1:] - g).exp().float()[..., None]).transpose(-1, -2) @ v    # [B, H, n, dk, dv]
    if init is None:
        init = q.new_zeros((B, H, dk, dv))
    G = torch.nn.functional.pad(g[..., -1].cumsum(-1), (1, 0))      # log decay from the start to each chunk
    carried = torch.cat([init[:, :, None], add], 2).flatten(3)      # state n = sum over m <= n of decay(m -> n) carried m
    after = torch.ones(n + 1, n + 1, dtype=torch.bool, device=q.device).triu(1)
    weight = (G[..., :, None] - G[..., None, :]).masked_fill(after, -math.inf).exp().float()
    states = (weight @ carried).unflatten(-1, (dk, dv))             # [B, H, n + 1, dk, dv]
    o = o + (q * g.exp().float()[..., None]) @ states[:, :, :-1]
    o = o.movedim(1, 3).flatten(1, 2)[:, :T]
    return o, states[:, :, -1]


def _plain_lin(q, k, v, la, init, cu):
    """fp32 o and final state from fp32 inputs (la fp64)."""
    if la.dim() == 1:
        la = la.expand(q.shape[:3])
    if cu is None:
        return _chunk_form(q, k, v, la, init)
    at, longest = _slots(cu, len(cu) - 1, 0, q.device)
    q, k, v, la = (_grid(x, at, len(cu) - 1, longest) for x in (q, k, v, la))
    o, final = _chunk_form(q, k, v, la, init)
    return o.flatten(0, 1)[at][None], final


def _plain_lin_fwd(st):
    dt = st["q"].dtype
    o, final = _plain_lin(st["q"].float(), st["k"].float(), st["v"].float(), st["log_alpha"].double(),
                          st["init"], st["cu"])
    return o.to(dt), final


def _plain_lin_bwd(st):
    dt = st["q"].dtype
    q, k, v = (st[x].float().requires_grad_() for x in ("q", "k", "v"))
    la = st["log_alpha"].double().requires_grad_()
    B, H, dk, dv = st["d_final"].shape
    init = (st["init"].clone() if st["init"] is not None else q.new_zeros((B, H, dk, dv))).requires_grad_()
    o, final = _plain_lin(q, k, v, la, init, st["cu"])
    got = torch.autograd.grad([o, final], [q, k, v, la, init], [st["d_o"].float(), st["d_final"]])
    return [x.to(dt) for x in got[:4]] + [got[4]]


def _plain_lin_decode(st):
    q, k, v, la = (st[x].float() for x in ("q", "k", "v", "log_alpha"))
    s = la.exp()[..., None, None] * st["state"] + k[..., :, None] * v[..., None, :]
    st["state"].copy_(s)
    return (q[..., None] * s).sum(-2).to(st["q"].dtype), st["state"]


def _angles(st):
    a = st["positions"].double()[:, None] * st["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _plain_norm_rope_one(x, w, cos, sin, rot, interleaved):
    y = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w
    r, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, rest], -1)


def _plain_norm_rope(st):
    c, dt = st["case"], st["q"].dtype
    cos, sin = _angles(st)
    return [_plain_norm_rope_one(st[x].float(), st[w].float(), cos, sin, c["rot"], c["interleaved"]).to(dt)
            for x, w in (("q", "wq"), ("k", "wk"))]


def _plain_norm_rope_bwd(st):
    c, dt, wdt = st["case"], st["q"].dtype, st["wq"].dtype
    cos, sin = _angles(st)
    q, k, wq, wk = (st[x].float().requires_grad_() for x in ("q", "k", "wq", "wk"))
    y = [_plain_norm_rope_one(x, w, cos, sin, c["rot"], c["interleaved"]) for x, w in ((q, wq), (k, wk))]
    dq, dk, dwq, dwk = torch.autograd.grad(y, [q, k, wq, wk], [st["d_q"].float(), st["d_k"].float()])
    return dq.to(dt), dk.to(dt), dwq.to(wdt), dwk.to(wdt)


# ---- one pass ------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        import kimi_delta_attention_30_b200 as kda
        if op == "lin_fwd":
            return kda.linear_chunk_fwd(state["q"], state["k"], state["v"], state["log_alpha"],
                                        init_state=state["init"], cu_seqlens=state["cu"])
        if op == "lin_bwd":
            return kda.linear_chunk_bwd(state["q"], state["k"], state["v"], state["log_alpha"], state["d_o"],
                                        init_state=state["init"], d_final_state=state["d_final"],
                                        cu_seqlens=state["cu"])
        if op == "lin_decode":
            return kda.linear_decode_step(state["q"], state["k"], state["v"], state["log_alpha"],
                                          state["state"]), state["state"]
        args = (state["q"], state["k"], state["wq"], state["wk"], state["positions"], state["inv_freq"])
        inter = state["case"]["interleaved"]
        if op == "norm_rope":
            return kda.qk_norm_rope(*args, eps=EPS, interleaved=inter)
        return kda.qk_norm_rope_bwd(*args, state["d_q"], state["d_k"], eps=EPS, interleaved=inter)
    return {"lin_fwd": _plain_lin_fwd, "lin_bwd": _plain_lin_bwd, "lin_decode": _plain_lin_decode,
            "norm_rope": _plain_norm_rope, "norm_rope_bwd": _plain_norm_rope_bwd}[op](state)


def _tokens(case):
    """Tokens of a lin_fwd / lin_bwd case."""
    return sum(_lengths(case)) if case["packed"] else case["B"] * case["T"]


def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("lin_fwd", "lin_bwd"):
        H, dk, dv = case["H"], case["dk"], case["dv"]
        tok, state = _tokens(case) * H, case["B"] * H * dk * dv
        la = tok * e if case["decay"] == "token" else 4 * H
        # the recurrence itself: decay and write the state, read it with the query
        if op == "lin_fwd":
            return {"bytes": tok * (2 * dk + 2 * dv) * e + la + 4 * state * (2 if case["init"] else 1),
                    "flops": tok * 4 * dk * dv}
        # q, k, v, d_o in and dq, dk, dv out; the states of both directions in the products
        return {"bytes": tok * (4 * dk + 3 * dv) * e + 2 * la + 4 * state * (3 if case["init"] else 2),
                "flops": tok * 10 * dk * dv}
    if op == "lin_decode":
        nh, dk, dv = case["B"] * case["H"], case["dk"], case["dv"]
        return {"bytes": nh * (8 * dk * dv + (2 * dk + 2 * dv) * e) + (nh * e if case["decay"] == "token" else 4 * case["H"]),
                "flops": nh * 5 * dk * dv}
    rows, d = case["B"] * case["T"] * (case["Hq"] + case["Hk"]), case["d"]
    w = 2 * d * (2 if case["wdtype"] == "bf16" else 4) + 2 * case["rot"] + 4 * case["B"] * case["T"]
    if op == "norm_rope":
        return {"bytes": rows * d * 2 * e + w, "flops": rows * d * 7}
    return {"bytes": rows * d * 3 * e + 2 * w, "flops": rows * d * 16}


# ---- values in 64 bits ---------------------------------------------------------

def _per_token(st):
    """fp64 inputs of the recurrence as [sequences, longest, H, ...], and the mask of real tokens."""
    names = [x for x in ("q", "k", "v", "d_o") if x in st]
    x = {n: st[n].double() for n in names}
    a = st["log_alpha"].double().exp()
    x["a"] = a if a.dim() == 3 else a.expand(st["q"].shape[:3])
    if st["cu"] is None:
        return x, None
    n = [b - a for a, b in zip(st["cu"][:-1], st["cu"][1:])]
    mask = torch.arange(max(n), device="cuda")[None] < torch.tensor(n, device="cuda")[:, None]
    out = {}
    for name, t in x.items():
        g = torch.full((len(n), max(n)) + t.shape[2:], 1.0 if name == "a" else 0.0, dtype=torch.float64, device="cuda")
        g[mask] = t[0]
        out[name] = g
    return out, mask


def _packed(x, mask):
    return x if mask is None else x[mask][None]


def _start(st, x):
    B, _, H, dk = x["q"].shape
    if st["init"] is not None:
        return st["init"].double().clone()
    return torch.zeros(B, H, dk, x["v"].shape[-1], dtype=torch.float64, device="cuda")


def _exact_fwd(st):
    x, mask = _per_token(st)
    s = _start(st, x)
    o = torch.empty_like(x["v"])
    for t in range(o.shape[1]):
        s.mul_(x["a"][:, t, :, None, None]).addcmul_(x["k"][:, t, :, :, None], x["v"][:, t, :, None, :])
        torch.matmul(x["q"][:, t, :, None, :], s, out=o[:, t, :, None, :])
    return _packed(o, mask), s


def _exact_bwd(st):
    x, mask = _per_token(st)
    q, k, v, a, do = (x[n] for n in ("q", "k", "v", "a", "d_o"))
    T, every = q.shape[1], 32
    s, kept = _start(st, x), []
    for t in range(T):
        if t % every == 0:
            kept.append(s.clone())
        s.mul_(a[:, t, :, None, None]).addcmul_(k[:, t, :, :, None], v[:, t, :, None, :])
    ds = st["d_final"].double().clone()
    dq, dk, dv, dla = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a)
    for b in reversed(range(len(kept))):
        t0, t1 = b * every, min(T, (b + 1) * every)
        before = [kept[b]]
        for t in range(t0, t1):
            before.append(before[-1] * a[:, t, :, None, None] + k[:, t, :, :, None] * v[:, t, :, None, :])
        for t in reversed(range(t0, t1)):
            ds.addcmul_(q[:, t, :, :, None], do[:, t, :, None, :])
            dq[:, t] = (before[t - t0 + 1] @ do[:, t, :, :, None])[..., 0]
            dk[:, t] = (ds @ v[:, t, :, :, None])[..., 0]
            dv[:, t] = (k[:, t, :, None, :] @ ds)[..., 0, :]
            dla[:, t] = a[:, t] * (ds * before[t - t0]).sum((-1, -2))
            ds.mul_(a[:, t, :, None, None])
    return [_packed(y, mask) for y in (dq, dk, dv, dla)] + [ds]


def _exact_decode(st):
    s = st["state"].double() * st["log_alpha"].double().exp()[..., None, None]
    s = s + torch.einsum("nhk,nhv->nhkv", st["k"].double(), st["v"].double())
    return torch.einsum("nhk,nhkv->nhv", st["q"].double(), s), s


def _turn(st):
    """The rotations as complex numbers [tokens, 1, rot / 2]."""
    a = st["positions"].double()[:, None, None] * st["inv_freq"].double()
    return torch.polar(torch.ones_like(a), a)


def _to_complex(x, rot, interleaved):
    r = x[..., :rot]
    pair = r.unflatten(-1, (rot // 2, 2)) if interleaved else r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
    return torch.view_as_complex(pair.contiguous())


def _from_complex(z, x, rot, interleaved):
    pair = torch.view_as_real(z)
    r = (pair if interleaved else pair.transpose(-1, -2)).flatten(-2)
    return torch.cat([r, x[..., rot:]], -1)


def _exact_norm_rope(st):
    c = st["case"]
    out = []
    for x, w in (("q", "wq"), ("k", "wk")):
        t = st[x].double()
        y = t / torch.sqrt((t ** 2).sum(-1, keepdim=True) / t.shape[-1] + EPS) * st[w].double()
        out.append(_from_complex(_to_complex(y, c["rot"], c["interleaved"]) * _turn(st), y, c["rot"], c["interleaved"]))
    return out


def _exact_norm_rope_bwd(st):
    c = st["case"]
    dx, dw = [], []
    for x, w, d in (("q", "wq", "d_q"), ("k", "wk", "d_k")):
        t, dy, wt = st[x].double(), st[d].double(), st[w].double()
        back = _to_complex(dy, c["rot"], c["interleaved"]) * _turn(st).conj()   # a rotation's gradient turns back
        g = _from_complex(back, dy, c["rot"], c["interleaved"])
        r = 1.0 / torch.sqrt((t ** 2).sum(-1, keepdim=True) / t.shape[-1] + EPS)
        dw.append((g * t * r).sum((0, 1)))
        h = g * wt
        dx.append(r * h - t * r ** 3 * (h * t).sum(-1, keepdim=True) / t.shape[-1])
    return dx + dw


def exact(case, seed):
    op = case["op"]
    if op in ("lin_fwd", "lin_bwd") and case["T"] * (12 if op == "lin_bwd" else 3) > 250_000:
        return None                       # token by token, it would take too long
    if op == "lin_bwd" and case["B"] * case["H"] * case["dk"] * case["dv"] * 8 * (33 + case["T"] / 32) > 6e10:
        return None                       # the kept states would not fit
    st = prepare(case, seed)
    return {"lin_fwd": _exact_fwd, "lin_bwd": _exact_bwd, "lin_decode": _exact_decode,
            "norm_rope": _exact_norm_rope, "norm_rope_bwd": _exact_norm_rope_bwd}[op](st)
