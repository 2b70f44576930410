"""Calls with `stream=`: their outputs and workspaces are theirs, whatever the
current stream does with memory that it frees before or takes afterwards."""
import pytest
import torch

from depth_wise_attention_gb300 import attnres

pytestmark = pytest.mark.gpu

N, S, T, D, H = 8, 4, 600, 1024, 4


def tensors(out):
    return [t for t in (out if isinstance(out, (tuple, list)) else [out]) if t is not None]


def calls():
    g = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    f32 = torch.float32
    A = attnres
    x, p, f = normal(N, T, D), normal(T, D), normal(T, D)
    w, gain, lse, lse_h = normal(S, D, dtype=f32) * 0.1, 1 + normal(D, dtype=f32) * 0.1, normal(T, dtype=f32), normal(H, T, dtype=f32)
    wh = w.view(S, H, D // H)
    dout = normal(S, T, D)
    cache = A.attnres_cache_quant(x, A.CACHE_FP4)
    ks = (2, 4, 8)
    cw, mq, mw = normal(D * sum(ks), dtype=f32) * 0.1, normal(4, D, dtype=f32) * 0.1, normal(4 * D, 4, dtype=f32) * 0.1
    return {
        "cache_quant": lambda s: A.attnres_cache_quant(x, A.CACHE_FP8, stream=s),
        "cache_dequant": lambda s: A.attnres_cache_dequant(cache, A.CACHE_FP4, D, stream=s),
        "cache_read": lambda s: A.attnres_cache_read(cache, A.CACHE_FP4, w, stream=s),
        "phase2_norm_q8": lambda s: A.attnres_phase2_norm_q8(x[0], lse, p, w[0], gain, f=f, want_h=True, stream=s),
        "norm_bwd": lambda s: A.attnres_norm_bwd(p, f, gain, stream=s),
        "full_fwd": lambda s: A.attnres_full_fwd(x, w[0], stream=s),
        "block_phase1": lambda s: A.attnres_block_phase1(x, w, stream=s),
        "block_phase2_update_merge": lambda s: A.attnres_block_phase2_update_merge(p, f, x[0], lse, w[0], stream=s),
        "mhar_phase2_merge": lambda s: A.mhar_phase2_merge(x[0], lse_h, p, wh[0], stream=s),
        "read_bwd": lambda s: A.attnres_read_bwd(x, w, dout, stream=s),
        "block_phase1_bwd": lambda s: A.attnres_block_phase1_bwd(x, w, dout, lse.expand(S, T).contiguous(), stream=s),
        "block_phase2_bwd": lambda s: A.attnres_block_phase2_bwd(x[0], lse, p, w[0], f, stream=s),
        "mhar_read_bwd": lambda s: A.mhar_read_bwd(x, wh, dout, stream=s),
        "mhar_fwd": lambda s: A.mhar_fwd(x, wh, want_lse=True, stream=s),
        "msar_expand_fwd_ws": lambda s: A.msar_expand_fwd_ws(x, ks, cw, mq, mix_w=mw, stream=s),
    }


@pytest.fixture(scope="module")
def cases():
    return calls()


NAMES = ["cache_quant", "cache_dequant", "cache_read", "phase2_norm_q8", "norm_bwd", "full_fwd", "block_phase1",
         "block_phase2_update_merge", "mhar_phase2_merge", "read_bwd", "block_phase1_bwd", "block_phase2_bwd", "mhar_read_bwd",
         "mhar_fwd", "msar_expand_fwd_ws"]
SIZES = [T * 4, D * 4, T * D * 2, S * T * D * 2, N * T * D * 2, N * T * D, 1 << 21, 1 << 22, 1 << 23, 1 << 24, 1 << 25]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_a_stream(cases, name):
    call, side = cases[name], torch.cuda.Stream()
    want = [t.clone() for t in tensors(call(None))]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # the current stream has work queued on memory that it has freed already
    old = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
    torch.cuda._sleep(20_000_000)
    for t in old:
        t.fill_(0xa5)
    del old, t
    # ... and the call's own stream is behind, so that its kernels run when the current one has taken new memory
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
    got = call(side)
    new = [torch.full((n,), 0x5a, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
    torch.cuda.synchronize()
    got = tensors(got)
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    for t in new:
        assert (t == 0x5a).all()
