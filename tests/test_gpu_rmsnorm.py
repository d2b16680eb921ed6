"""GPU parity of rmsnorm_quantize: the residual stream, codes and scales bit
for bit against the oracle, for every format and block size, odd row counts,
strided and in-place buffers, rows that are zero or not finite.

Why exact equality can be asked: every step is one pinned fp32 operation
except the sum of squares, which both sides form in fp64 (relative error
below K 2^-53); its effect on inv is a changed rounding only within that
distance of a rounding border, for about one row in 10^6."""
import numpy as np
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from oracle import formats as F, norm as NM
from helpers import dev_bf16, host_bits, need_gpu, log

pytestmark = pytest.mark.gpu
EPS = 1e-6
FMTS = ["int8", "bf16", "mxfp4", "mxfp8"]


def laplace(rng, M, K, mult=2.0):
    x = rng.laplace(size=(M, K)).astype(np.float32) * mult
    x[:, rng.integers(0, K, size=max(1, K // 200))] *= 30
    return F.f32_to_bf16(x)


def equal_out(got, o, fmt, rows=slice(None)):
    if fmt == "bf16":
        q = host_bits(got.q)[rows]
        fin = o["finite"]
        assert np.array_equal(q[fin], o["q"][fin])
        assert np.isnan(F.bf16_to_f32(q[~fin])).all()
        return
    q, s = got.q.cpu().numpy()[rows], got.scales.cpu().numpy()[rows]
    assert np.array_equal(q, o["q"]), np.argwhere(q != o["q"])[:4]
    assert np.array_equal(s, o["scales"], equal_nan=fmt == "int8"), np.argwhere(s != o["scales"])[:4]


def check(M, K, b, fmt, res=True, gain=True, seed=0):
    rng = np.random.Generator(np.random.PCG64(1000 + seed))
    log(f"rmsnorm M={M} K={K} b={b} {fmt} res={res} gain={gain}")
    x, r = laplace(rng, M, K), laplace(rng, M, K) if res else None
    w = (1 + 0.2 * rng.standard_normal(K)).astype(np.float32) if gain else None
    got, s = V.rmsnorm_quantize(dev_bf16(x), torch.from_numpy(w).cuda() if gain else None,
                                dev_bf16(r) if res else None, EPS, b, fmt)
    torch.cuda.synchronize()
    o = NM.rmsnorm_quantize(x, r, w, EPS, b, fmt)
    equal_out(got, o, fmt)
    if res:
        assert np.array_equal(host_bits(s), o["r"])
    else:
        assert s is None


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K,b", [
    (1, 64, 64), (1, 32, 32), (5, 64, 16), (37, 96, 32), (3, 128, 128), (2, 256, 256), (17, 256, 64), (9, 384, 128),
    (65, 512, 64), (4, 768, 256), (33, 1920, 64), (257, 1920, 128), (1, 3072, 64), (130, 3072, 256), (7, 4096, 32),
    (3, 4160, 64), (2, 7680, 64), (5, 12288, 256), (2, 16384, 16), (1100, 192, 64), (2049, 3072, 64)])
def test_sizes(M, K, b, fmt):
    need_gpu()
    check(M, K, b, fmt, seed=M + K + b)


@pytest.mark.parametrize("K,b", [(16, 16), (48, 16), (80, 16), (2000, 16)])
@pytest.mark.parametrize("fmt", ["int8", "bf16"])
def test_widths_below_a_block_of_32(K, b, fmt):
    need_gpu()
    for M in (1, 3, 70):
        check(M, K, b, fmt, seed=K)


@pytest.mark.parametrize("res,gain", [(False, False), (False, True), (True, False)])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,K", [(6, 1920), (1500, 3072), (3, 192), (3, 8192)])
def test_without_residual_or_gain(M, K, fmt, res, gain):
    need_gpu()
    check(M, K, 64, fmt, res, gain, seed=7)


@pytest.mark.parametrize("fmt", FMTS)
def test_zero_tiny_and_bad_rows(fmt):
    """Zero rows, rows around eps and far below the smallest code scale,
    one NaN, one infinity, an addition that overflows: only those rows are
    marked."""
    need_gpu()
    rng = np.random.Generator(np.random.PCG64(3))
    for M, K in ((9, 320), (1030, 320), (9, 128)):
        log(f"bad rows M={M} K={K} {fmt}")
        x, r = laplace(rng, M, K), laplace(rng, M, K)
        x[0], r[0] = 0, 0
        x[1] = F.f32_to_bf16((rng.standard_normal(K) * 1e-3).astype(np.float32))
        r[1] = 0
        x[2] = F.f32_to_bf16((rng.standard_normal(K) * 1e-36).astype(np.float32))
        r[2] = 0
        x[3, K - 1] = 0x7FC0                     # NaN
        r[5, 0] = 0xFF80                         # -inf
        x[7, 3] = r[7, 3] = 0x7F60                # 2.98e38: the sum overflows
        got, s = V.rmsnorm_quantize(dev_bf16(x), None, dev_bf16(r), EPS, 64, fmt)
        torch.cuda.synchronize()
        o = NM.rmsnorm_quantize(x, r, None, EPS, 64, fmt)
        assert list(np.nonzero(~o["finite"])[0]) == [3, 5, 7]
        equal_out(got, o, fmt)
        ok = np.isfinite(F.bf16_to_f32(o["r"]))
        assert np.array_equal(host_bits(s)[ok], o["r"][ok])


@pytest.mark.parametrize("fmt", FMTS)
def test_strides_and_reused_outputs(fmt):
    """Rows inside wider tensors, outputs of an earlier call reused, the
    bytes around the strided sum untouched."""
    need_gpu()
    rng = np.random.Generator(np.random.PCG64(4))
    M, K = 45, 640
    x, r = laplace(rng, M, K), laplace(rng, M, K)
    wide = torch.full((M, 3 * K + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :K] = dev_bf16(x)
    wide[:, K + 8:2 * K + 8] = dev_bf16(r)
    o = NM.rmsnorm_quantize(x, r, None, EPS, 64, fmt)
    out, _ = V.rmsnorm_quantize(dev_bf16(r), None, None, EPS, 64, fmt)
    q0 = out.q
    got, s = V.rmsnorm_quantize(wide[:, :K], None, wide[:, K + 8:2 * K + 8], EPS, 64, fmt, out=out,
                                sum_out=wide[:, 2 * K + 8:])
    torch.cuda.synchronize()
    assert got.q.data_ptr() == q0.data_ptr()
    equal_out(got, o, fmt)
    h = host_bits(wide)
    assert np.array_equal(h[:, 2 * K + 8:], o["r"]) and np.array_equal(h[:, :K], x)
    assert (F.bf16_to_f32(h[:, K:K + 8]) == 7.0).all() and np.array_equal(h[:, K + 8:2 * K + 8], r)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("M,K", [(3, 3072), (2000, 3072), (40, 128), (5, 9216)])
def test_stream_updated_in_place(which, M, K):
    need_gpu()
    rng = np.random.Generator(np.random.PCG64(6))
    x, r = laplace(rng, M, K), laplace(rng, M, K)
    xd, rd = dev_bf16(x), dev_bf16(r)
    dst = xd if which == "x" else rd
    log(f"in place {which} M={M} K={K}")
    got, s = V.rmsnorm_quantize(xd, None, rd, EPS, 64, "mxfp8", sum_out=dst)
    torch.cuda.synchronize()
    assert s.data_ptr() == dst.data_ptr()
    o = NM.rmsnorm_quantize(x, r, None, EPS, 64, "mxfp8")
    equal_out(got, o, "mxfp8")
    assert np.array_equal(host_bits(dst), o["r"])


@pytest.mark.parametrize("M,K,b", [(9, 256, 128), (300, 512, 256), (1024, 2064, 16), (1023, 3056, 16), (1500, 2560, 64),
                                   (5, 5120, 256), (6, 6144, 64), (6, 6160, 16), (3, 8192, 128), (3, 10240, 64),
                                   (70, 1040, 16), (3000, 64, 32), (900, 48, 16)])
def test_borders_of_the_lane_counts(M, K, b):
    need_gpu()
    for fmt in ("int8", "bf16") if K % 32 else FMTS:
        check(M, K, b, fmt, seed=M)


@pytest.mark.parametrize("fmt", ["int8", "mxfp8", "bf16"])
@pytest.mark.parametrize("M,K", [(17776, 3072), (21000, 2048), (12000, 6144), (700000, 64)])
def test_large_inputs_are_their_parts(M, K, fmt):
    """Above 256 MB the inputs are read past the cache: the bits are those
    of the same rows in small calls."""
    need_gpu()
    log(f"large {M} x {K} {fmt}")
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.randn(M, K, device="cuda", generator=g) * 3).bfloat16()
    r = (torch.randn(M, K, device="cuda", generator=g) * 3).bfloat16()
    w = 1 + 0.1 * torch.randn(K, device="cuda", generator=g)
    whole, s = V.rmsnorm_quantize(x, w, r, EPS, 64, fmt)
    for a in range(0, M, M // 5 + 1):
        b = min(M, a + M // 5 + 1)
        part, t = V.rmsnorm_quantize(x[a:b], w, r[a:b], EPS, 64, fmt)
        assert torch.equal(part.q.view(torch.uint8), whole.q[a:b].view(torch.uint8)) and torch.equal(t, s[a:b])
        if fmt != "bf16":
            assert torch.equal(part.scales, whole.scales[a:b])


def test_no_rows():
    need_gpu()
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    out, s = V.rmsnorm_quantize(x, None, x, fmt="mxfp8")
    assert out.q.shape == (0, 128) and s.shape == (0, 128)


def test_matches_norm_then_hadamard_quantize():
    """The one-pass result is hadamard_quantize's when y is exact in bf16:
    rows of +-2^k whose mean square is 1 (eps far below it)."""
    need_gpu()
    rng = np.random.Generator(np.random.PCG64(8))
    x = dev_bf16(F.f32_to_bf16(rng.choice([-1.0, 1.0], size=(50, 1024)).astype(np.float32)))
    for fmt in FMTS:
        got, _ = V.rmsnorm_quantize(x, None, None, 1e-30, 64, fmt)
        want = V.hadamard_quantize(x, 64, fmt)
        assert torch.equal(got.q, want.q)
        if fmt != "bf16":
            assert torch.equal(got.scales, want.scales)
