"""The largest sizes that the norm, few-row and grouped calls document: rows,
features and K at or just below their limits, on contents that repeat (with a
period that is prime), so that small calls give the expected values."""
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from helpers import log, need_gpu

pytestmark = pytest.mark.gpu
P = 997


def rand(rows, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, K, device="cuda", generator=g).bfloat16()


def periodic(t, rows):
    """t's rows repeated to so many."""
    return t.repeat(rows // t.shape[0] + 1, 1)[:rows]


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
def test_norm_rows_past_one_dimension_of_the_launch(fmt):
    """More than 2^22 workgroups of 32 rows: the rows fold over the launch's
    second dimension; elements past 2^31."""
    need_gpu()
    M, K = 134300000, 16
    assert M > (1 << 22) * 32 and M * K > 1 << 31
    x, r = rand(P, K, 1), rand(P, K, 2)
    want, s = V.rmsnorm_quantize(x, None, r, had_block=16, fmt=fmt)
    got, t = V.rmsnorm_quantize(periodic(x, M), None, periodic(r, M), had_block=16, fmt=fmt)
    torch.cuda.synchronize()
    whole = M // P * P
    for big, small in [(got.q, want.q), (t, s)] + ([(got.scales[:, None], want.scales[:, None])] if fmt == "int8" else []):
        assert (big[:whole].view(-1, P, small.shape[1]) == small).all() and torch.equal(big[whole:], small[:M - whole])


@pytest.mark.parametrize("which", ["w4a16", "mx", "grouped"])
def test_most_features(which):
    """2^26 - 1 features."""
    need_gpu()
    N, K, M = (1 << 26) - 1, 128, 2
    log(f"{which} N={N}")
    a = rand(M, K, 3)
    if which == "w4a16":
        w = V.hadamard_quantize(rand(P, K, 4), 64, "nvfp4")
        big = V.NVFP4Tensor(periodic(w.q, N), periodic(w.scales, N), w.ts)
        call = lambda v: V.qgemv_w4a16(V.BF16Tensor(a), v)     # noqa: E731
    else:
        am = V.hadamard_quantize(a, 64, "mxfp8")
        w = V.hadamard_quantize(rand(P, K, 4), 64, "mxfp4")
        big = V.MXTensor(periodic(w.q, N), periodic(w.scales, N), "mxfp4")
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        call = (lambda v: V.qgemv_mx(am, v)) if which == "mx" else (lambda v: V.qgemm_mx_grouped(am, v, off))
    want, y = call(w), call(big)
    torch.cuda.synchronize()
    whole = N // P * P
    assert (y[:, :whole].view(M, -1, P) == want[:, None]).all() and torch.equal(y[:, whole:], want[:, :N - whole])


@pytest.mark.parametrize("kind", ["w4a16", "w4a8", "mxfp8", "mxfp4", "grouped"])
def test_longest_rows(kind):
    """K = 2^24 of elements 0 and +-1: every partial sum is an integer of at
    most 2^24 and so exact in fp32."""
    need_gpu()
    K, N, M = 1 << 24, 17, 3
    log(f"K = 2^24 {kind}")
    g = torch.Generator(device="cuda").manual_seed(5)
    A = torch.randint(-1, 2, (M, K), device="cuda", generator=g, dtype=torch.int8)
    W = torch.randint(-1, 2, (N, K), device="cuda", generator=g, dtype=torch.int8)
    want = torch.stack([torch.stack([(A[m] * W[n]).sum(dtype=torch.int64) for n in range(N)]) for m in range(M)])

    def e2m1(v):                                              # +-1 is code 2, the sign bit 8
        c = torch.where(v == 0, 0, torch.where(v > 0, 2, 10)).to(torch.uint8)
        return c[:, 0::2] | (c[:, 1::2] << 4)

    mx = kind not in ("w4a16", "w4a8")
    if mx:
        w = V.MXTensor(e2m1(W), torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda"), "mxfp4")
        one = torch.full((M, K // 32), 127, dtype=torch.uint8, device="cuda")
        e4m3 = torch.where(A == 0, 0, torch.where(A > 0, 0x38, 0xB8)).to(torch.uint8)
        a = V.MXTensor(e2m1(A), one, "mxfp4") if kind == "mxfp4" else V.MXTensor(e4m3, one, "mxfp8")
        if kind == "grouped":
            off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
            y = V.qgemm_mx_grouped(a, w, off, None, "f32")
            assert torch.equal(V.qgemm_mx_grouped(a, w, off).double(), want.double().bfloat16().double())
        else:
            y = V.qgemv_mx(a, w, None, "f32")
    else:
        w = V.NVFP4Tensor(e2m1(W), torch.full((N, K // 16), 0x38, dtype=torch.uint8, device="cuda"),
                          torch.ones(2, device="cuda"))
        y = (V.qgemv_w4a16(V.BF16Tensor(A.bfloat16()), w, None, "f32") if kind == "w4a16" else
             V.qgemv_w4a8(V.INT8Tensor(A, torch.ones(M, device="cuda")), w, None, "f32"))
    torch.cuda.synchronize()
    assert torch.equal(y.double(), want.double())
