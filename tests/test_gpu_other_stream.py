"""The wrappers on a stream that is not the current one: their workspaces and
converted copies belong to that stream, and arguments that the caller drops keep
their memory until it has read them."""

import pytest
import torch

from long_context_compressed_overlapped_b200 import api, synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cases():
    g = torch.Generator(device=DEV).manual_seed(3)

    def normal(*s, dt=torch.bfloat16):
        return torch.randn(*s, generator=g, device=DEV).to(dt)
    B, n, m, d, w = 2, 64, 4, 512, 16
    pos = torch.tensor([511, 300], device=DEV)                              # (int64: converted)
    a, b, za, zb, bias = normal(B, n, d), normal(B, n, d), normal(B, n, d), normal(B, n, d), normal(m, d)
    yield "csa_compress", lambda x, **kw: api.csa_compress(x[0], x[1], x[2], x[3], x[4], x[4], m, gain=x[5], rope_dims=64, **kw), \
        [a, b, za, zb, bias, normal(d)]
    codes, scale = synth.quantize_e4m3_rows(normal(B, 3000, 128))
    yield "indexer_topk", lambda x, **kw: api.indexer_topk(x[0], x[1], x[2], x[3], m, 64, kI_scale=x[4], **kw), \
        [normal(B, 3, 64, 128), normal(B, 3, 64), codes, torch.full((B, 3), 12000, device=DEV), scale.double()]
    yield "indexer_topk by name", lambda x, **kw: api.indexer_topk(qI=x[0], w=x[1], kI=x[2], q_pos=x[3], m=m, k=64, kI_scale=x[4], **kw), \
        [normal(B, 3, 64, 128), normal(B, 3, 64), codes, torch.full((B, 3), 12000, device=DEV), scale.double()]
    yield "compressed_attn_prefill", lambda x, **kw: api.compressed_attn_prefill("hca", x[0], x[1], x[2], x[3], m=m, w=w, rope_dims=64,
                                                                                 q_gain=x[4], **kw), \
        [normal(1, n, 64, d), normal(1, n // m, d), normal(1, n, d), normal(64), normal(d)]
    yield "compressed_attn_decode", lambda x, **kw: api.compressed_attn_decode("hca", x[0], x[1], x[2], x[3], x[4], m=m, rope_dims=64,
                                                                               q_gain=x[5], **kw), \
        [normal(B, 64, d), pos, normal(B, 200, d), normal(B, w, d), normal(64), normal(d)]

    def step(x, **kw):
        ring, kv = x[5].clone(), torch.zeros(B, 200, d, device=DEV, dtype=torch.bfloat16)
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        api.decode_compress("csa", x[0], tuple(x[1:5]), ring, kv, m=m, bias_a=x[6], bias_b=x[6], kv_gain=x[7], rope_dims=64, **kw)
        step.held = ring, kv
        return kv
    yield "decode_compress", step, [pos, normal(B, d), normal(B, d), normal(B, d), normal(B, d), normal(B, 2 * m, 4, d), bias, normal(d)]
    ci = torch.stack([torch.arange(8, device=DEV, dtype=torch.int32)[None]] * 2)
    yield "cp_topk_merge", lambda x, **kw: api.cp_topk_merge(x[0], x[1], [0, 100], 0, **kw)[0], [ci, normal(2, 1, 8, dt=torch.float32)]
    yield "cp_attn_merge", lambda x, **kw: api.cp_attn_merge(x[0], x[1], x[2], H=4, d=64, rope_dims=16, **kw), \
        [normal(2, B, 2 * 4 + 4 * 64, dt=torch.float32).abs(), normal(4), pos]


@pytest.mark.parametrize("name", ["csa_compress", "indexer_topk", "indexer_topk by name", "compressed_attn_prefill", "compressed_attn_decode", "decode_compress",
                                  "cp_topk_merge", "cp_attn_merge"])
def test_call_on_another_stream(name):
    call, args = next((c, a) for n, c, a in cases() if n == name)
    want = call(args)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    slow = torch.randn(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(10):
            slow = slow @ slow * 1e-3
    mine = [x.clone() for x in args]
    torch.cuda.current_stream().synchronize()
    sizes = [x.numel() * x.element_size() for x in mine]
    got = call(mine, stream=st)
    del mine
    junk = [torch.zeros(s, dtype=torch.uint8, device=DEV) for s in sizes for _ in range(8)]     # (what is free on the current stream)
    junk += [torch.zeros(1 << e, dtype=torch.uint8, device=DEV) for e in range(9, 27) for _ in range(4)]
    st.synchronize()
    assert torch.equal(got, want)
    del junk
    with pytest.raises(ValueError):
        call([x.cpu() for x in args])
    assert api.device_error() == 0
