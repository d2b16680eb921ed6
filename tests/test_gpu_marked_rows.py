"""Rows that the norm marks as not finite, through every product that reads
them: INT8 scale NaN with codes 0, MX scale byte 0xFF with codes 0, BF16 NaNs
make each of the row's products NaN, and no other row's bits change."""
import numpy as np
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from helpers import log, need_gpu

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def rand(rows, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, K, device="cuda", generator=g).bfloat16()


def part(t, lo, hi):
    if isinstance(t, V.BF16Tensor):
        return V.BF16Tensor(t.q[lo:hi])
    if isinstance(t, V.INT8Tensor):
        return V.INT8Tensor(t.q[lo:hi], t.scales[lo:hi])
    return V.MXTensor(t.q[lo:hi], t.scales[lo:hi], t.fmt)


def normed(M, K, fmt, bad, seed=1):
    """(rows without, rows with) a NaN, an infinity or a sum that overflows
    in the rows `bad`, as the norm writes them."""
    x, r = rand(M, K, seed), rand(M, K, seed + 1)
    clean, _ = V.rmsnorm_quantize(x, None, r, fmt=fmt)
    for n, row in enumerate(bad):
        if n % 3 == 0:
            x[row, K - 1] = NAN
        elif n % 3 == 1:
            r[row, 0] = -INF
        else:
            x[row, 5] = r[row, 5] = 3e38
    marked, _ = V.rmsnorm_quantize(x, None, r, fmt=fmt)
    if fmt != "bf16":
        assert (marked.q[bad] == 0).all()
        assert torch.isnan(marked.scales[bad]).all() if fmt == "int8" else (marked.scales[bad] == 0xFF).all()
    return clean, marked


def check(y, clean, bad):
    torch.cuda.synchronize()
    keep = torch.ones(y.shape[0], dtype=torch.bool)
    keep[bad] = False
    assert torch.isnan(y[bad]).all(), f"{int((~torch.isnan(y[bad])).sum())} products of marked rows are not NaN"
    assert torch.isfinite(y[keep]).all() and torch.equal(y[keep], clean[keep])


CALL = {"bf16": V.qgemv_w4a16, "int8": V.qgemv_w4a8, "mxfp8": V.qgemv_mx, "mxfp4": V.qgemv_mx}


@pytest.mark.parametrize("fmt", list(CALL))
@pytest.mark.parametrize("M,bad", [(1, [0]), (3, [1]), (4, [0, 3]), (5, [4]), (16, [0, 7, 15]), (17, [16]), (32, [0, 15, 16, 31])])
def test_few_rows(fmt, M, bad):
    need_gpu()
    for N, K in ((40, 256), (33, 1024), (64, 4096)):
        log(f"marked rows {fmt} M={M} N={N} K={K}")
        a, m = normed(M, K, fmt, bad)
        w = V.hadamard_quantize(rand(N, K, 3), 64, "mxfp4" if fmt.startswith("mx") else "nvfp4")
        bias = torch.randn(N, device="cuda")
        for od in ("bf16", "f32"):
            check(CALL[fmt](m, w, bias, od), CALL[fmt](a, w, bias, od), bad)


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,N,K", [
    ([3, 0, 4, 2], 80, 256), ([12, 9], 40, 7680),         # few rows an expert
    ([40, 0, 33, 20], 200, 512),                          # small tiles
    ([1900, 0, 2196], 2700, 256)])                        # large tiles
def test_rows_by_expert(fmt, counts, N, K):
    need_gpu()
    T = sum(counts)
    log(f"marked rows by expert {fmt} counts={counts} N={N} K={K}")
    bad = [0, T // 2, T - 1]
    a, m = normed(T, K, fmt, bad)
    w = V.hadamard_quantize(rand(len(counts) * N, K, 3), 64, "mxfp4")
    bias = torch.randn(len(counts), N, device="cuda")
    off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()
    for od in ("bf16", "f32"):
        check(V.qgemm_mx_grouped(m, w, off, bias, od), V.qgemm_mx_grouped(a, w, off, bias, od), bad)


@pytest.mark.parametrize("fmt", ["int8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("M", [3, 9, 32])
def test_one_bad_scale_under_ordinary_codes(fmt, M):
    """A NaN scale (INT8) or a single block's 0xFF (MX) whatever the codes."""
    need_gpu()
    for N, K in ((40, 288 if fmt != "int8" else 272), (64, 4096)):
        g = torch.Generator(device="cuda").manual_seed(M)
        x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
        b = 32 if fmt != "int8" else 16
        a = V.hadamard_quantize(x, b, fmt)
        w = V.hadamard_quantize(rand(N, K, 3), b, "nvfp4" if fmt == "int8" else "mxfp4")
        clean = CALL[fmt](a, w, None, "f32").clone()
        if fmt == "int8":
            a.scales[1] = NAN
        else:
            a.scales[1, K // 32 - 1] = 0xFF
        check(CALL[fmt](a, w, None, "f32"), clean, [1])


@pytest.mark.parametrize("fmt", ["mxfp8", "mxfp4"])
def test_a_bad_weight_scale_makes_its_feature_nan(fmt):
    """0xFF among the weights' scales: that feature is NaN in every row, also
    over zero codes, and no other feature changes."""
    need_gpu()
    for M, N, K in ((2, 40, 256), (11, 33, 1024), (30, 64, 512)):
        a = V.hadamard_quantize(rand(M, K, 5), 64, fmt)
        w = V.hadamard_quantize(rand(N, K, 6), 64, "mxfp4")
        off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
        calls = [lambda: V.qgemv_mx(a, w, None, "f32"), lambda: V.qgemm_mx_grouped(a, w, off, None, "f32"),
                 lambda: V.qgemm_mx_grouped(a, w, off)]
        clean = [c().clone() for c in calls]
        w.scales[7, 3] = 0xFF
        w.scales[N - 1, K // 32 - 1] = 0xFF
        w.q[N - 1] = 0
        for c, was in zip(calls, clean):
            y = c()
            check(y.t(), was.t(), [7, N - 1])
