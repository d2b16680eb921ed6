"""GPU parity of the products of few rows (qgemv_w4a16, qgemv_w4a8, qgemv_mx)
and of rows grouped by expert (qgemm_mx_grouped), and the norm feeding them.

Tolerances (helpers.assert_elementwise): the products are exact, so an
element errs by the fp32 additions of K terms and a few roundings of the
scale and bias, at most 2 (K + 4) 2^-24 of the sum of absolute terms, and by
half a bf16 step (2^-8 relative) where the output is bf16."""
import numpy as np
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from oracle import formats as F, gemm as G, norm as NM, quant as Q
from helpers import (assert_elementwise, bf16_values, dev_bf16, host_bits, need_gpu, log, terms_mx, terms_w4a8,
                     terms_w4a16)

pytestmark = pytest.mark.gpu


def rng_of(*k):
    return np.random.Generator(np.random.PCG64(list(k)))


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def weights(rng, N, K, kind):
    """Codes and scales of random weights, made by the oracle."""
    w = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    if kind == "mx":
        q, s = Q.mx_quantize(w, "e2m1")
        return (q, s), V.MXTensor(dev(q), dev(s), "mxfp4")
    q, s, ts = Q.nvfp4_quantize(w)
    return (q, s, ts[1]), V.NVFP4Tensor(dev(q), dev(s), dev(np.array(ts, np.float32)))


def acts(rng, M, K, kind):
    x = (rng.laplace(size=(M, K)) * 2).astype(np.float32)
    x[:, rng.integers(0, K, size=max(1, K // 200))] *= 30
    if kind == "w4a16":
        b = F.f32_to_bf16(x)
        return (b,), V.BF16Tensor(dev_bf16(b))
    if kind == "w4a8":
        q, s = Q.int8_quantize(x)
        return (q, s), V.INT8Tensor(dev(q), dev(s))
    q, s = Q.mx_quantize(x, Q.MX_ELEM[kind])
    return (q, s), V.MXTensor(dev(q), dev(s), kind)


def reference(kind, a, w, bias):
    """float64 Y and the sums of absolute terms."""
    if kind == "w4a16":
        return G.qgemm_w4a16(a[0], *w, bias, "f32")[0], terms_w4a16(a[0], *w, bias)
    if kind == "w4a8":
        return G.qgemm_w4a8(*a, *w, bias, "f32")[0], terms_w4a8(*a, *w, bias)
    return G.qgemm_mx(*a, kind, *w, bias, "f32")[0], terms_mx(*a, kind, *w, bias)


CALL = {"w4a16": V.qgemv_w4a16, "w4a8": V.qgemv_w4a8, "mxfp8": V.qgemv_mx, "mxfp4": V.qgemv_mx}


def values(y):
    return bf16_values(host_bits(y)) if y.dtype == torch.bfloat16 else y.cpu().numpy()


def check_gemv(kind, M, N, K, bias=True, seed=0):
    rng = rng_of(M, N, K, seed)
    log(f"gemv {kind} M={M} N={N} K={K} bias={bias}")
    ah, ad = acts(rng, M, K, kind)
    wh, wd = weights(rng, N, K, "mx" if kind.startswith("mx") else "nv")
    bh = rng.standard_normal(N).astype(np.float32) if bias else None
    want, terms = reference(kind, ah, wh, bh)
    for od in ("bf16", "f32"):
        y = CALL[kind](ad, wd, None if bh is None else dev(bh), od)
        torch.cuda.synchronize()
        assert_elementwise(values(y), want, terms, K, od, f"{kind} {od}")
    return ad, wd, want, terms


KINDS = ["w4a16", "w4a8", "mxfp8", "mxfp4"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 24, 31, 32])
def test_gemv_rows(kind, M):
    need_gpu()
    check_gemv(kind, M, 77, 640, bias=M % 2 == 0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,K", [(1, 32), (1, 3072), (15, 64), (16, 128), (17, 96), (33, 160), (65, 1920), (127, 2080),
                                 (1920, 1920), (200, 7680), (31, 12288), (4097, 256), (3072, 512)])
@pytest.mark.parametrize("M", [1, 7, 32])
def test_gemv_sizes(kind, N, K, M):
    need_gpu()
    check_gemv(kind, M, N, K, seed=1)


@pytest.mark.parametrize("kind", ["w4a16", "w4a8"])
@pytest.mark.parametrize("K", [16, 48, 80, 144, 1936, 3088])
def test_gemv_widths_of_half_a_load(kind, K):
    """K a multiple of 16 and not of 32: a row's last 8 code bytes stand
    alone, and rows start 8 bytes off a 16-byte boundary."""
    need_gpu()
    for M, N in ((1, 5), (6, 37), (32, 18)):
        check_gemv(kind, M, N, K, seed=2)


@pytest.mark.parametrize("kind", KINDS)
def test_gemv_output_in_a_wider_tensor(kind):
    need_gpu()
    rng = rng_of(11)
    M, N, K = 6, 50, 256
    ah, ad = acts(rng, M, K, kind)
    wh, wd = weights(rng, N, K, "mx" if kind.startswith("mx") else "nv")
    want, terms = reference(kind, ah, wh, None)
    for od, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        wide = torch.full((M + 2, N + 5), 7.0, dtype=dt, device="cuda")
        y = CALL[kind](ad, wd, None, od, y=wide[1:M + 1, 3:N + 3])
        torch.cuda.synchronize()
        assert_elementwise(values(y.contiguous()), want, terms, K, od, kind)
        wide[1:M + 1, 3:N + 3] = 7.0
        assert (wide == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gemv_weights_inside_larger_ones(kind):
    """Rows cut out of stacked weights: scales that start at odd bytes where
    K is no multiple of 128, and row views where it is."""
    need_gpu()
    rng = rng_of(14)
    for N, K, skip in ((40, 96, 1), (33, 160, 3), (24, 1920, 5), (24, 640, 2)):
        ah, ad = acts(rng, 5, K, kind)
        wh, wd = weights(rng, N, K, "mx" if kind.startswith("mx") else "nv")
        g = K // (32 if kind.startswith("mx") else 16)
        codes = torch.zeros((N + 16) * K // 2, dtype=torch.uint8, device="cuda")
        codes[8 * K:8 * K + N * K // 2] = wd.q.flatten()              # 16 rows of K / 2 bytes in
        scales = torch.zeros((N + 16) * g, dtype=torch.uint8, device="cuda")
        scales[skip * g:(skip + N) * g] = wd.scales.flatten()
        q, s = codes[8 * K:8 * K + N * K // 2].view(N, K // 2), scales[skip * g:(skip + N) * g].view(N, g)
        w = V.MXTensor(q, s, "mxfp4") if kind.startswith("mx") else V.NVFP4Tensor(q, s, wd.ts)
        assert torch.equal(CALL[kind](ad, w, None, "f32"), CALL[kind](ad, wd, None, "f32"))


@pytest.mark.parametrize("kind", KINDS)
def test_gemv_rows_that_are_not_finite(kind):
    """A NaN (bf16), a NaN scale (INT8) or an 0xFF scale byte (MX) makes its
    row of Y NaN; the other rows keep their bits."""
    need_gpu()
    rng = rng_of(12)
    for M, N, K in ((3, 40, 288), (20, 33, 1024), (5, 64, 4096)):
        log(f"bad row {kind} M={M}")
        _, ad = acts(rng, M, K, kind)
        _, wd = weights(rng, N, K, "mx" if kind.startswith("mx") else "nv")
        clean = CALL[kind](ad, wd, None, "f32").clone()
        if kind == "w4a16":
            ad.q[1, 0] = float("nan")
            ad.q[M - 1, K - 1] = float("inf")
        elif kind == "w4a8":
            ad.scales[1] = float("nan")
            ad.scales[M - 1] = float("nan")
        else:
            ad.scales[1, 0] = 0xFF
            ad.scales[M - 1, K // 32 - 1] = 0xFF
        y = CALL[kind](ad, wd, None, "f32")
        torch.cuda.synchronize()
        bad = torch.zeros(M, dtype=torch.bool)
        bad[1] = bad[M - 1] = True
        assert (~torch.isfinite(y[bad])).all() and torch.equal(y[~bad], clean[~bad])


def test_gemv_agrees_with_the_gemm_of_its_name():
    need_gpu()
    rng = rng_of(13)
    M, N, K = 8, 256, 512
    for kind, big in (("w4a16", V.qgemm_w4a16), ("w4a8", V.qgemm_w4a8), ("mxfp4", V.qgemm_mx)):
        ah, ad = acts(rng, M, K, kind)
        wh, wd = weights(rng, N, K, "mx" if kind.startswith("mx") else "nv")
        _, terms = reference(kind, ah, wh, None)
        assert_elementwise(values(CALL[kind](ad, wd, None, "f32")), values(big(ad, wd, None, "f32")), 2 * terms, K, "f32")


# ------------------------------------------------------------------ grouped
def cut_off(a_q, a_s, w_q, w_s):
    """What the block-scaled matrix instruction may drop of MXFP8 x MXFP4
    sums (bf16 output of many rows).  Measured on the instruction, with one
    large, one cancelling and one small product: it adds the products of 8
    consecutive k after cutting each, towards zero, at 2^-13 of the power of
    two below the largest of the 8; products of other eights, other blocks
    and the running sum are not cut against each other.  Of 8 products at
    most 7 lose bits (the largest has 5 significant bits or fewer, so it
    keeps them all), each less than 2^-13 max|p|, so the sum of an eight is
    off by less than 7 * 2^-13 max|p|."""
    A = np.abs(Q.mx_dequantize(a_q, a_s, "e4m3"))
    W = np.abs(Q.mx_dequantize(w_q, w_s, "e2m1"))
    out = np.zeros((A.shape[0], W.shape[0]))
    for k in range(0, A.shape[1], 8):
        m = A[:, k, None] * W[None, :, k]
        for i in range(k + 1, k + 8):
            np.maximum(m, A[:, i, None] * W[None, :, i], out=m)
        out += m
    return 7 * 2.0 ** -13 * out


def check_grouped(afmt, counts, N, K, bias=True, front=0, back=0, ods=("bf16", "f32"), seed=0, sample=None):
    rng = rng_of(N, K, len(counts), seed)
    E, T = len(counts), front + sum(counts) + back
    log(f"grouped {afmt} counts={counts if E < 20 else (E, sum(counts))} N={N} K={K} front={front} back={back}")
    ah, ad = acts(rng, T, K, afmt)
    wh, wd = weights(rng, E * N, K, "mx")
    bh = rng.standard_normal((E, N)).astype(np.float32) if bias else None
    off = np.concatenate([[front], front + np.cumsum(counts)]).astype(np.int32)
    want, cov = G.qgemm_mx_grouped(*ah, afmt, *wh, off, bh)
    terms, cut = np.zeros_like(want), np.zeros_like(want)
    for e in range(E):
        r, w = slice(off[e], off[e + 1]), slice(e * N, (e + 1) * N)
        if off[e + 1] > off[e]:
            if afmt == "mxfp8" and "bf16" in ods:
                cut[r] = cut_off(ah[0][r], ah[1][r], wh[0][w], wh[1][w])
            terms[r] = terms_mx(ah[0][r], ah[1][r], afmt, wh[0][w], wh[1][w], None if bh is None else bh[e])
    for od in ods:
        y = torch.full((T, N), 7.0, dtype=torch.bfloat16 if od == "bf16" else torch.float32, device="cuda")
        V.qgemm_mx_grouped(ad, wd, dev(off), None if bh is None else dev(bh), od, y=y)
        torch.cuda.synchronize()
        v = values(y)
        assert (v[~cov] == 7.0).all(), "a row outside every group was written"
        if cov.any():
            # the cut is passed as terms that give it at the bound's 2 (K + 4) 2^-24
            more = cut[cov] / (2 * (K + 4) * 2.0 ** -24) if od == "bf16" else 0
            assert_elementwise(v[cov], want[cov], terms[cov] + more, K, od, f"grouped {afmt} {od}")


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", [
    [1], [0, 1], [1, 0, 0, 2], [3, 0, 5, 1, 0, 7, 16, 2], [17, 33, 0, 31, 32], [64, 1, 65, 0, 63], [0, 0, 0], [130, 2],
    [100, 100, 90, 110], [257, 255, 1], [300, 0, 20, 511]])
def test_grouped_counts(afmt, counts):
    need_gpu()
    check_grouped(afmt, counts, 96, 256, bias=len(counts) % 2 == 0)


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("N,K", [(1, 128), (7, 128), (64, 384), (130, 512), (257, 640), (520, 1024), (192, 1920), (31, 3072)])
@pytest.mark.parametrize("counts", [[2, 9, 0, 4], [70, 33, 90], [300, 280]])
def test_grouped_sizes(afmt, N, K, counts):
    need_gpu()
    check_grouped(afmt, counts, N, K, front=3, back=5)


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("K", [7168, 7296, 12288, 14336, 14464])
def test_grouped_long_rows(afmt, K):
    """K around the borders where the few-row kernel takes K in two turns
    and where it gives way to tiles."""
    need_gpu()
    check_grouped(afmt, [3, 0, 12, 1], 40, K)


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts", [[12], [13], [12, 12], [13, 13], [191], [192], [191, 191], [192, 192], [0, 0, 0, 40],
                                    [200, 1, 1, 1], [1, 1, 500]])
def test_grouped_borders_of_the_kernels(afmt, counts):
    need_gpu()
    check_grouped(afmt, counts, 136, 640, back=2)


@pytest.mark.parametrize("kind", ["mxfp8", "mxfp4"])
def test_scales_far_from_one(kind):
    """Block scales of 2^-60 and 2^50 against weights of 2^40 and 2^-30."""
    need_gpu()
    rng = rng_of(26)
    for T, E in ((5, 1), (40, 2), (500, 2)):
        N, K = 48, 512
        (aq, as_), ad = acts(rng, T, K, kind)
        (wq, ws), wd = weights(rng, E * N, K, "mx")
        as_ = as_.copy()
        ws = ws.copy()
        as_[:, 0::2] -= 60
        ws[:, 0::2] += 40
        as_[:, 1::2] += 50
        ws[:, 1::2] -= 30
        ad.scales.copy_(dev(as_))
        wd.scales.copy_(dev(ws))
        off = np.array([0, T] if E == 1 else [0, T // 3, T], np.int32)
        want, _ = G.qgemm_mx_grouped(aq, as_, kind, wq, ws, off)
        y = V.qgemm_mx_grouped(ad, wd, dev(off), None, "f32")
        torch.cuda.synchronize()
        for e in range(E):
            r, w = slice(off[e], off[e + 1]), slice(e * N, (e + 1) * N)
            t = terms_mx(aq[r], as_[r], kind, wq[w], ws[w], None)
            assert_elementwise(values(y)[r], want[r], t, K, "f32", kind)
        if T <= 32 and E == 1:
            assert_elementwise(values(V.qgemv_mx(ad, wd, None, "f32")), want, t, K, "f32", kind)


def test_grouped_weights_of_4_gb():
    """An expert whose codes reach past 32-bit offsets: its last features
    have the values that they have as an expert of their own.  (Both sums are
    exact up to fp32 and the instruction's cut, 3.4e-5 of the norm here; one
    bf16 step, 2^-7, covers a rounding that falls the other way.)"""
    need_gpu()
    K, N, T = 1 << 18, 32800, 200
    assert N * K // 2 >= 1 << 32
    g = torch.Generator(device="cuda").manual_seed(4)
    w = V.MXTensor(torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda", generator=g),
                   torch.randint(120, 124, (N, K // 32), dtype=torch.uint8, device="cuda", generator=g), "mxfp4")
    a = V.hadamard_quantize((torch.randn(T, K, device="cuda", generator=g)).bfloat16(), 64, "mxfp8")
    off = dev(np.array([0, T], np.int32))
    y = V.qgemm_mx_grouped(a, w, off).float()
    for lo, hi in ((0, 70), (N - 90, N)):
        part = V.MXTensor(w.q[lo:hi].contiguous(), w.scales[lo:hi].contiguous(), "mxfp4")
        z = V.qgemm_mx_grouped(a, part, off).float()
        torch.cuda.synchronize()
        tol = 2.0 ** -7 * z.abs() + 40 * 3.4e-5 * z.pow(2).mean().sqrt()
        assert ((y[:, lo:hi] - z).abs() <= tol).all()


def test_grouped_many_experts():
    need_gpu()
    c = rng_of(21).integers(0, 4, size=300).tolist()
    check_grouped("mxfp8", c, 48, 128)
    check_grouped("mxfp4", [0] * 299 + [3], 48, 128)


def test_grouped_bad_offsets_stay_inside():
    """Offsets that fall, are negative or pass T reach nothing outside y:
    each counts as the largest up to there, inside [0, T]."""
    need_gpu()
    rng = rng_of(22)
    N, K, T = 64, 256, 40
    ah, ad = acts(rng, T, K, "mxfp8")
    wh, wd = weights(rng, 4 * N, K, "mx")
    for off in ([-5, 10, 4, 12, 40], [0, 50, 60, 70, 80], [0, 10, 1 << 30, -(1 << 31), 39], [40, 0, 0, 0, 0]):
        log(f"offsets {off}")
        clean = np.maximum.accumulate(np.clip(off, 0, T))
        guard = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
        V.qgemm_mx_grouped(ad, wd, dev(np.array(off, np.int32)), y=guard[1:T + 1])
        want = torch.full((T + 2, N), 7.0, dtype=torch.bfloat16, device="cuda")
        V.qgemm_mx_grouped(ad, wd, dev(clean.astype(np.int32)), y=want[1:T + 1])
        torch.cuda.synchronize()
        assert torch.equal(guard, want)


def test_grouped_output_strides():
    need_gpu()
    rng = rng_of(23)
    for counts, N, K in (([5, 9], 48, 128), ([200, 120], 264, 256)):
        T = sum(counts)
        ah, ad = acts(rng, T, K, "mxfp8")
        wh, wd = weights(rng, 2 * N, K, "mx")
        off = dev(np.array([0, counts[0], T], np.int32))
        for od, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
            want = V.qgemm_mx_grouped(ad, wd, off, None, od)
            for pad, shift in ((8, 0), (5, 3)):
                wide = torch.full((T, N + pad), 7.0, dtype=dt, device="cuda")
                y = V.qgemm_mx_grouped(ad, wd, off, None, od, y=wide[:, shift:N + shift])
                torch.cuda.synchronize()
                assert torch.equal(y, want)
                wide[:, shift:N + shift] = 7.0
                assert (wide == 7.0).all()


def test_grouped_rows_that_are_not_finite():
    need_gpu()
    rng = rng_of(24)
    for counts in ([3, 4, 2], [150, 140], [400, 390]):
        T, N, K = sum(counts), 80, 256
        _, ad = acts(rng, T, K, "mxfp8")
        _, wd = weights(rng, len(counts) * N, K, "mx")
        off = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        for od in ("bf16", "f32"):
            clean = V.qgemm_mx_grouped(ad, wd, off, None, od).clone()
            keep = ad.scales.clone()
            ad.scales[1, 0] = 0xFF
            ad.scales[T - 1, K // 32 - 1] = 0xFF
            y = V.qgemm_mx_grouped(ad, wd, off, None, od)
            torch.cuda.synchronize()
            bad = torch.zeros(T, dtype=torch.bool)
            bad[1] = bad[T - 1] = True
            assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], clean[~bad])
            ad.scales.copy_(keep)


def test_grouped_equal_experts_are_one_product():
    """Rows in two groups of the same weights give the bits of one group
    where both calls take the same kernel, and sums of another order (twice
    the bound of one) where 24 rows of one expert and 12 of each of two do
    not."""
    need_gpu()
    rng = rng_of(25)
    for T, cut, same in ((12, 5, True), (24, 9, False), (600, 256, True)):
        N, K = 128, 512
        (aq, as_), ad = acts(rng, T, K, "mxfp8")
        (q, s), one = weights(rng, N, K, "mx")
        two = V.MXTensor(dev(np.concatenate([q, q])), dev(np.concatenate([s, s])), "mxfp4")
        a = V.qgemm_mx_grouped(ad, one, dev(np.array([0, T], np.int32)), None, "f32")
        b = V.qgemm_mx_grouped(ad, two, dev(np.array([0, cut, T], np.int32)), None, "f32")
        if same:
            assert torch.equal(a, b)
        assert_elementwise(values(a), values(b), 2 * terms_mx(aq, as_, "mxfp8", q, s, None), K, "f32")


# -------------------------------------------------------- the run together
def chain(x, res, gain, w8, w16, wmx, wexp, off):
    """Norm to each format, the products that read it, rows by expert."""
    a8, s = V.rmsnorm_quantize(x, gain, res, fmt="int8")
    a16, _ = V.rmsnorm_quantize(x, gain, res, fmt="bf16")
    amx, _ = V.rmsnorm_quantize(x, gain, res, fmt="mxfp8")
    return [s, V.qgemv_w4a8(a8, w8), V.qgemv_w4a16(a16, w16, None, "f32"), V.qgemv_mx(amx, wmx),
            V.qgemm_mx_grouped(amx, wexp, off)]


def chain_inputs(seed, M=24, K=512, N=320):
    rng = rng_of(seed)
    x, r = (F.f32_to_bf16((rng.laplace(size=(M, K)) * 2).astype(np.float32)) for _ in range(2))
    gain = (1 + 0.1 * rng.standard_normal(K)).astype(np.float32)
    off = np.array([0, 5, 5, 20, M], np.int32)
    wh8, w8 = weights(rng, N, K, "nv")
    whm, wm = weights(rng, N, K, "mx")
    whe, we = weights(rng, 4 * N, K, "mx")
    return (x, r, gain, wh8, whm, whe, off), (dev_bf16(x), dev_bf16(r), dev(gain), w8, w8, wm, we, dev(off))


def test_chain_against_the_oracle():
    need_gpu()
    (x, r, gain, wh8, whm, whe, off), d = chain_inputs(31)
    got = chain(*d)
    torch.cuda.synchronize()
    K = x.shape[1]
    o8, o16, om = (NM.rmsnorm_quantize(x, r, gain, 1e-6, 64, f) for f in ("int8", "bf16", "mxfp8"))
    assert np.array_equal(host_bits(got[0]), o8["r"])
    assert_elementwise(values(got[1]), G.qgemm_w4a8(o8["q"], o8["scales"], *wh8, None, "f32")[0],
                       terms_w4a8(o8["q"], o8["scales"], *wh8, None), K, "bf16")
    assert_elementwise(values(got[2]), G.qgemm_w4a16(o16["q"], *wh8, None, "f32")[0],
                       terms_w4a16(o16["q"], *wh8, None), K, "f32")
    tm = terms_mx(om["q"], om["scales"], "mxfp8", *whm, None)
    assert_elementwise(values(got[3]), G.qgemm_mx(om["q"], om["scales"], "mxfp8", *whm, None, "f32")[0], tm, K, "bf16")
    want, _ = G.qgemm_mx_grouped(om["q"], om["scales"], "mxfp8", *whe, off)
    N = whm[0].shape[0]
    te = np.concatenate([terms_mx(om["q"][a:b], om["scales"][a:b], "mxfp8", whe[0][e * N:(e + 1) * N],
                                  whe[1][e * N:(e + 1) * N], None)
                         for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a])
    cut = np.concatenate([cut_off(om["q"][a:b], om["scales"][a:b], whe[0][e * N:(e + 1) * N], whe[1][e * N:(e + 1) * N])
                          for e, (a, b) in enumerate(zip(off[:-1], off[1:])) if b > a])
    assert_elementwise(values(got[4]), want, te + cut / (2 * (K + 4) * 2.0 ** -24), K, "bf16")


_FIRST_CALLS_UNDER_CAPTURE = r"""
import sys
import torch
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import test_gpu_few_rows as T
ins = T.chain_inputs(51, M=30)[1]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = T.chain(*ins)                      # the process's first calls
for _ in range(3):
    g.replay()
    torch.cuda.synchronize()
    want = T.chain(*ins)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
print("ok")
"""


def test_first_calls_under_capture():
    """Nothing that a first call sets up is missing from a graph that was
    captured before any eager call (in a fresh process)."""
    need_gpu()
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS_UNDER_CAPTURE, root], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout[-2000:] + r.stderr[-2000:]


def test_native_and_python_marshalling_agree(monkeypatch):
    """The native entry takes the ordinary calls (given outputs among them)
    and the Python path gives the same bits; what the native entry declines
    (strided outputs, refused sizes, wrong types) the Python path does or
    refuses."""
    need_gpu()
    from video_diffusion_transformer_block_amd import ops as O
    assert O._fast is not None, "the native entry is not built"
    ins = chain_inputs(62)[1]
    fast = [t.clone() for t in chain(*ins)]
    x, res, gain, w8, _, wm, we, off = ins
    a8, _ = V.rmsnorm_quantize(x, gain, res)
    y = torch.full((x.shape[0], w8.q.shape[0]), 7.0, dtype=torch.bfloat16, device="cuda")
    assert V.qgemv_w4a8(a8, w8, y=y) is y and torch.equal(y, fast[1])
    calls = []

    class Spy:
        def __getattr__(self, name):
            def call(*args):
                r = getattr(O_fast, name)(*args)
                calls.append((name, r is not None))
                return r
            return call

    O_fast = O._fast
    monkeypatch.setattr(O, "_fast", Spy())
    again = chain(*ins)
    assert all(torch.equal(a, b) for a, b in zip(again, fast))
    assert calls == [("norm", True)] * 3 + [("gemv", True)] * 3 + [("grouped", True)]
    calls.clear()
    wide = torch.empty((x.shape[0], y.shape[1] + 4), dtype=torch.bfloat16, device="cuda")
    assert torch.equal(V.qgemv_w4a8(a8, w8, y=wide[:, :y.shape[1]]), fast[1]) and calls == [("gemv", False)]
    for bad in (lambda: V.qgemv_w4a8(a8, w8, torch.zeros(3, device="cuda")), lambda: V.qgemv_w4a8(a8, w8, None, "f16"),
                lambda: V.rmsnorm_quantize(x[:, :24]), lambda: V.rmsnorm_quantize(x, gain[:5]),
                lambda: V.rmsnorm_quantize(x, gain, None, sum_out=x), lambda: V.rmsnorm_quantize(x.float()),
                lambda: V.qgemm_mx_grouped(V.rmsnorm_quantize(x, fmt="mxfp8")[0], we, off.long())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: V.rmsnorm_quantize(x, eps=0.0), lambda: V.rmsnorm_quantize(x, had_block=48),
                lambda: V.qgemv_w4a8(V.INT8Tensor(a8.q.repeat(2, 1), a8.scales.repeat(2)), w8)):
        with pytest.raises(V.VdtqError):
            bad()
    monkeypatch.setattr(O, "_fast", None)
    slow = chain(*ins)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(slow, fast))


def test_chain_from_two_threads():
    """Two host threads, a stream each, the same operands read by both: the
    bits of a lone call."""
    need_gpu()
    import threading
    ins = chain_inputs(61)[1]
    want = [t.clone() for t in chain(*ins)]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = chain(*ins)
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append(k)
        except Exception as e:                   # reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_chain_in_graphs_and_on_two_streams():
    """Two captured graphs of the chain (one of them with changed inputs and
    row counts between replays), eager calls in between, and the chain on two
    streams at once: every result has the bits of a lone eager call."""
    need_gpu()
    ins = [list(chain_inputs(41)[1]), list(chain_inputs(42)[1])]
    want = [[t.clone() for t in chain(*i)] for i in ins]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in ins:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(chain(*i))
        graphs.append(g)
    for rep in range(3):
        for k in (0, 1):
            log(f"replay {rep} of graph {k}")
            graphs[k].replay()
            eager = chain(*ins[1 - k])
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs[k], want[k]))
            assert all(torch.equal(a, b) for a, b in zip(eager, want[1 - k]))
    other = dev(np.array([0, 0, 11, 11, 24], np.int32))
    ins[0][0].copy_(ins[1][0])
    ins[0][7].copy_(other)
    graphs[0].replay()
    torch.cuda.synchronize()
    now = chain(*ins[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], now))
    want[0] = [t.clone() for t in now]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [None, None]
    for rep in range(3):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = chain(*ins[k])
        torch.cuda.synchronize()
        for k in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(got[k], want[k]))


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("counts,N,K", [
    ([130, 126], 12288, 256), ([100, 0, 28], 9216, 128), ([400, 368], 1024, 512), ([1500, 4], 264, 128),
    ([3, 2200, 0, 41], 1000, 256), ([14, 13, 12, 20], 8200, 128)])
def test_grouped_where_either_tile_may_serve(afmt, counts, N, K):
    """Counts and sizes on both sides of the choice between the two tile
    sizes."""
    need_gpu()
    check_grouped(afmt, counts, N, K, front=1, back=2)


@pytest.mark.parametrize("counts,N,K", [
    ([12, 13], 100, 512), ([15, 17], 4100, 256), ([16], 70, 1152), ([17], 70, 1152), ([5, 0, 7], 4561, 5504),
    ([1, 0, 0, 1, 0, 0], 4619, 1280), ([9, 2], 40, 16384)])
def test_grouped_few_rows_in_many_workgroups(counts, N, K):
    """Both few-row kernels where a workgroup takes one, several or not all
    feature blocks, and K of one and of many turns."""
    need_gpu()
    check_grouped("mxfp8", counts, N, K, front=1, back=1)
