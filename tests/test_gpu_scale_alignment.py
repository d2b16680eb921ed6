"""Block scales that start at any byte, also where K is a multiple of 128 and
a row's scales are whole words: the few-row products read them in runs of any
alignment."""
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from helpers import log, need_gpu
from test_gpu_few_rows import CALL, KINDS, acts, rng_of, weights

pytestmark = pytest.mark.gpu


def shifted(s, by):
    """The same bytes, `by` past a 256-byte boundary, others around them."""
    big = torch.full((s.numel() + by + 8,), 0xFF, dtype=torch.uint8, device="cuda")
    v = big[by:by + s.numel()].view(s.shape)
    v.copy_(s)
    return v


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 37, 128), (3, 16, 640), (9, 50, 1920), (20, 33, 3072), (32, 17, 256)])
def test_scales_at_any_byte(kind, M, N, K):
    need_gpu()
    rng = rng_of(M, N, K)
    _, a = acts(rng, M, K, kind)
    _, w = weights(rng, N, K, "mx" if kind.startswith("mx") else "nv")
    want = CALL[kind](a, w, None, "f32")
    for by in (1, 2, 3, 4, 7):
        log(f"scales at {by} {kind} M={M} N={N} K={K}")
        if kind.startswith("mx"):
            b, v = V.MXTensor(a.q, shifted(a.scales, 8 - by), kind), V.MXTensor(w.q, shifted(w.scales, by), "mxfp4")
        else:
            b, v = a, V.NVFP4Tensor(w.q, shifted(w.scales, by), w.ts)
        assert torch.equal(CALL[kind](b, v, None, "f32"), want)
