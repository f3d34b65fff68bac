"""Tensors that a call writes in place count as modified for autograd."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _writes():
    """{name: (tensors the call writes, the call)}"""
    import kimi_delta_attention_30_b200 as kda
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.nn.functional.normalize(torch.randn(*s, generator=g), dim=-1).to(BF).cuda()
    q, k, v = r(1, 70, 2, 128), r(1, 70, 2, 128), r(1, 70, 2, 128)
    la, lah = (-torch.rand(1, 70, 2, 128, generator=g)).to(BF).cuda(), (-torch.rand(1, 70, 2, generator=g)).to(BF).cuda()
    beta = torch.full((1, 70, 2), 0.5, dtype=BF, device="cuda")
    w = torch.ones(128, dtype=BF, device="cuda")
    o, o1 = torch.empty_like(v), torch.empty_like(v[:, 0])
    s = lambda: torch.zeros(1, 2, 128, 128, device="cuda")
    kg = tuple(torch.empty_like(t) for t in (q, k, v, la, beta)) + (s(),)
    lg = tuple(torch.empty_like(t) for t in (q, k, v, lah)) + (s(),)
    ng = tuple(torch.empty_like(t) for t in (q, k, w, w))
    st = [s() for _ in range(4)]
    cpu = [t.cpu() for t in (q, k, v, la, beta)]
    ho, hs = torch.empty(1, 70, 2, 128, dtype=BF), torch.empty(1, 2, 128, 128)
    M, F = kda.segment_map(q, k, v, la, beta)
    out = torch.empty(2, 1, 2, 128, 128, device="cuda")
    one = [t[:, 0].contiguous() for t in (q, k, v, la, beta, lah)]
    return dict(
        chunk_fwd=([o, st[0]], lambda: kda.chunk_fwd(q, k, v, la, beta, o=o, final_state=st[0])),
        chunk_fwd_noalloc=([o, st[0]], lambda: kda.chunk_fwd_noalloc(q, k, v, la, beta, o=o, final_state=st[0])),
        chunk_fwd_host=([ho, hs], lambda: kda.chunk_fwd_host(*cpu, [0, 70], o=ho, final_state=hs)),
        chunk_bwd=(list(kg), lambda: kda.chunk_bwd(q, k, v, la, beta, v, grads=kg)),
        segment_map=([M, F], lambda: kda.segment_map(q, k, v, la, beta, M=M, F=F)),
        compose_states=([out], lambda: kda.compose_states(M[None], F[None], out=out)),
        decode_step=([st[1], o1], lambda: kda.decode_step(*one[:5], st[1], o=o1)),
        linear_chunk_fwd=([o, st[2]], lambda: kda.linear_chunk_fwd(q, k, v, lah, o=o, final_state=st[2])),
        linear_chunk_bwd=(list(lg), lambda: kda.linear_chunk_bwd(q, k, v, lah, v, grads=lg)),
        linear_decode_step=([st[3], o1], lambda: kda.linear_decode_step(*one[:3], one[5], st[3], o=o1)),
        qk_norm_rope=([q, k], lambda: kda.qk_norm_rope(q, k, w, w, q_out=q, k_out=k)),
        qk_norm_rope_bwd=(list(ng), lambda: kda.qk_norm_rope_bwd(q, k, w, w, None, None, v, v, grads=ng)),
    )


NAMES = ["chunk_fwd", "chunk_fwd_noalloc", "chunk_fwd_host", "chunk_bwd", "segment_map", "compose_states", "decode_step",
         "linear_chunk_fwd", "linear_chunk_bwd", "linear_decode_step", "qk_norm_rope", "qk_norm_rope_bwd"]


@pytest.mark.parametrize("name", NAMES)
def test_written_tensors_are_noticed(cuda_ok, name):
    tensors, call = _writes()[name]
    leaf = torch.ones((), device=tensors[0].device, dtype=torch.float32, requires_grad=True)
    products = [leaf * t for t in tensors]      # each keeps t for its backward
    before = [t._version for t in tensors]
    call()
    assert all(t._version > v for t, v in zip(tensors, before))
    for y in products:
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_inference_tensors_are_written_too(cuda_ok):
    with torch.inference_mode():
        for name, (_, call) in _writes().items():
            call()
