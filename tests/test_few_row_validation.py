"""CPU tests of what rmsnorm_quantize, qgemv_* and qgemm_mx_grouped refuse,
at the C entry points (nothing is launched: every call fails or is a no-op)
and in the binding."""
import ctypes

import pytest
import torch

import video_diffusion_transformer_block_amd as V
from video_diffusion_transformer_block_amd import _lib as L
from video_diffusion_transformer_block_amd import ops as O
from test_ops_validation import mx, nv, stub, u8  # noqa: F401

FAKE = ctypes.c_void_p(0x100000)         # aligned, never dereferenced
FAKE2 = ctypes.c_void_p(0x900000)
FAKE3 = ctypes.c_void_p(0x1100000)
ODD = ctypes.c_void_p(0x100008)


def _norm(**kw):
    a = dict(x=FAKE, M=4, K=64, ldx=64, r=FAKE2, ldr=64, w=None, eps=1e-6, b=64, fmt=L.FMT_INT8,
             sum=ctypes.c_void_p(0x1900000), lds=64, q=FAKE3, s=ctypes.c_void_p(0x2100000))
    a.update(kw)
    return V.lib().rmsnorm_quantize(a["x"], a["M"], a["K"], a["ldx"], a["r"], a["ldr"], a["w"], a["eps"], a["b"],
                                    a["fmt"], a["sum"], a["lds"], a["q"], a["s"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), L.EINVAL), (dict(M=1 << 31), L.EINVAL), (dict(K=0), L.EINVAL), (dict(K=72, ldx=72), L.EINVAL),
    (dict(K=96, ldx=96), L.EINVAL), (dict(b=48), L.EINVAL), (dict(b=512, K=512), L.EINVAL), (dict(ldx=60), L.EINVAL),
    (dict(ldx=68), L.EINVAL), (dict(ldr=32), L.EINVAL), (dict(lds=66), L.EINVAL), (dict(fmt=9), L.EINVAL),
    (dict(fmt=L.FMT_NVFP4), L.EUNSUPPORTED), (dict(fmt=L.FMT_MXFP8, K=48, ldx=48, b=16), L.EINVAL),
    (dict(K=16448, ldx=16448, ldr=16448, lds=16448), L.EUNSUPPORTED), (dict(eps=0.0), L.EINVAL),
    (dict(eps=-1.0), L.EINVAL), (dict(eps=float("nan")), L.EINVAL), (dict(eps=float("inf")), L.EINVAL),
    (dict(x=None), L.EINVAL), (dict(q=None), L.EINVAL), (dict(s=None), L.EINVAL), (dict(x=ODD), L.EINVAL),
    (dict(q=ODD), L.EINVAL), (dict(w=ODD), L.EINVAL), (dict(r=None), L.EINVAL),
    # overlaps: the sum shifted into x by a row, in a column range of x's, over q; q over x
    (dict(sum=ctypes.c_void_p(0x100000 + 128)), L.EINVAL), (dict(sum=FAKE, lds=128), L.EINVAL),
    (dict(sum=ctypes.c_void_p(0x900000 + 2 * 32), ldr=128, lds=128), L.EINVAL),
    (dict(sum=FAKE3), L.EINVAL), (dict(q=FAKE), L.EINVAL), (dict(q=FAKE2), L.EINVAL), (dict(s=FAKE3), L.EINVAL),
    (dict(w=FAKE3), L.EINVAL), (dict(w=ctypes.c_void_p(0x1900000)), L.EINVAL),
])
def test_rmsnorm_rejects(kw, code):
    assert _norm(**kw) == code
    assert V.lib().vdtq_last_error()


def test_rmsnorm_empty_is_noop():
    assert _norm(M=0, x=None, q=None, s=None) == L.OK


def _gemv(fn, **kw):
    a = dict(fmt=L.FMT_MXFP8, aq=FAKE, as_=FAKE, wq=FAKE, ws=FAKE, wts=FAKE, bias=None, y=FAKE, ldy=64, od=0, M=8, N=64,
             K=64)
    a.update(kw)
    tail = (a["bias"], a["y"], a["ldy"], a["od"], a["M"], a["N"], a["K"], None)
    if fn == "w4a16":
        return V.lib().qgemv_w4a16(a["aq"], a["wq"], a["ws"], a["wts"], *tail)
    if fn == "w4a8":
        return V.lib().qgemv_w4a8(a["aq"], a["as_"], a["wq"], a["ws"], a["wts"], *tail)
    return V.lib().qgemv_mx(a["fmt"], a["aq"], a["as_"], a["wq"], a["ws"], *tail)


@pytest.mark.parametrize("fn", ["w4a16", "w4a8", "mx"])
@pytest.mark.parametrize("kw,code", [
    (dict(K=0), L.EINVAL), (dict(K=40), L.EINVAL), (dict(M=-1), L.EINVAL), (dict(N=-1), L.EINVAL), (dict(ldy=63), L.EINVAL),
    (dict(od=2), L.EINVAL), (dict(aq=None), L.EINVAL), (dict(wq=None), L.EINVAL), (dict(ws=None), L.EINVAL),
    (dict(y=None), L.EINVAL), (dict(aq=ODD), L.EINVAL), (dict(wq=ODD), L.EINVAL), (dict(M=33), L.EUNSUPPORTED),
    (dict(bias=ctypes.c_void_p(0x100002)), L.EINVAL), (dict(M=1 << 31), L.EINVAL),
    (dict(K=(1 << 24) + 128), L.EUNSUPPORTED), (dict(N=1 << 26, ldy=1 << 26), L.EUNSUPPORTED),
])
def test_qgemv_rejects(fn, kw, code):
    assert _gemv(fn, **kw) == code
    assert V.lib().vdtq_last_error()


def test_qgemv_format_rules():
    assert _gemv("mx", fmt=L.FMT_INT8) == L.EINVAL
    assert _gemv("mx", K=48) == L.EINVAL
    assert _gemv("w4a16", wts=None) == L.EINVAL and _gemv("w4a8", wts=None) == L.EINVAL
    odd = ctypes.c_void_p(0x100002)
    for fn in ("w4a16", "w4a8", "mx"):                       # scale runs need alignment, bytes do not
        assert _gemv(fn, K=128, ws=odd) == L.EINVAL
    assert _gemv("w4a16", K=256, ws=ctypes.c_void_p(0x100004)) == L.EINVAL and _gemv("mx", K=128, as_=odd) == L.EINVAL
    assert _gemv("w4a8", as_=None) == L.EINVAL and _gemv("mx", as_=None) == L.EINVAL
    for fn in ("w4a16", "w4a8", "mx"):
        assert _gemv(fn, M=0, aq=None) == L.OK and _gemv(fn, N=0, y=None) == L.OK


def _grp(**kw):
    a = dict(fmt=L.FMT_MXFP8, aq=FAKE, as_=FAKE, wq=FAKE, ws=FAKE, bias=None, off=FAKE, E=4, y=FAKE, ldy=64, od=0, T=8,
             N=64, K=128)
    a.update(kw)
    return V.lib().qgemm_mx_grouped(a["fmt"], a["aq"], a["as_"], a["wq"], a["ws"], a["bias"], a["off"], a["E"], a["y"],
                                    a["ldy"], a["od"], a["T"], a["N"], a["K"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(fmt=L.FMT_NVFP4), L.EINVAL), (dict(E=-1), L.EINVAL), (dict(E=65537), L.EINVAL), (dict(K=0), L.EINVAL),
    (dict(K=48), L.EINVAL), (dict(K=96), L.EUNSUPPORTED), (dict(K=(1 << 24) + 128), L.EUNSUPPORTED), (dict(T=-1), L.EINVAL), (dict(N=-1), L.EINVAL),
    (dict(ldy=10), L.EINVAL), (dict(od=3), L.EINVAL), (dict(off=None), L.EINVAL), (dict(aq=None), L.EINVAL),
    (dict(as_=None), L.EINVAL), (dict(wq=None), L.EINVAL), (dict(ws=None), L.EINVAL), (dict(y=None), L.EINVAL),
    (dict(aq=ODD), L.EINVAL), (dict(off=ctypes.c_void_p(0x100002)), L.EINVAL), (dict(T=(1 << 30) + 1), L.EUNSUPPORTED),
    (dict(N=1 << 26, ldy=1 << 26), L.EUNSUPPORTED), (dict(T=1 << 30, N=4096, ldy=4096), L.EUNSUPPORTED),
    (dict(T=1 << 24, N=8192, ldy=8192, od=1), L.EUNSUPPORTED),
    (dict(T=1 << 26, N=4096, ldy=4096, K=1 << 22), L.EUNSUPPORTED),
])
def test_grouped_rejects(kw, code):
    assert _grp(**kw) == code
    assert V.lib().vdtq_last_error()


def test_grouped_empty_is_noop():
    assert _grp(T=0, aq=None) == L.OK and _grp(N=0, y=None) == L.OK and _grp(E=0, wq=None, off=None) == L.OK


M, N, K = 8, 64, 128


def i8(m=M, k=K):
    return O.INT8Tensor(torch.zeros((m, k), dtype=torch.int8), torch.zeros(m))


def bf(m=M, k=K):
    return O.BF16Tensor(torch.zeros((m, k), dtype=torch.bfloat16))


OFF = torch.zeros(3, dtype=torch.int32)


def test_binding_passes_valid_buffers(stub):  # noqa: F811
    x = torch.zeros((M, K), dtype=torch.bfloat16)
    for fmt in ("int8", "bf16", "mxfp4", "mxfp8"):
        out, s = O.rmsnorm_quantize(x, torch.ones(K), x.clone(), fmt=fmt)
        assert s.shape == x.shape
        out2, s = O.rmsnorm_quantize(x, fmt=fmt, out=out)
        assert s is None and out2.q is out.q
    r = x.clone()
    assert O.rmsnorm_quantize(x, None, r, sum_out=r)[1] is r
    O.qgemv_w4a16(bf(), nv(N, K), torch.zeros(N))
    O.qgemv_w4a8(i8(), nv(N, K), y=torch.zeros((M, 2 * N), dtype=torch.bfloat16)[:, :N])
    O.qgemv_mx(mx(M, K, "mxfp8"), mx(N, K))
    assert O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), OFF, torch.zeros(2, N), "f32").shape == (M, N)
    assert stub.calls[-4:] == ["qgemv_w4a16", "qgemv_w4a8", "qgemv_mx", "qgemm_mx_grouped"]


BAD = {
    "x f32": lambda x: O.rmsnorm_quantize(x.float()),
    "x 1-D": lambda x: O.rmsnorm_quantize(x[0]),
    "x column stride": lambda x: O.rmsnorm_quantize(x.t()),
    "fmt": lambda x: O.rmsnorm_quantize(x, fmt="nvfp4"),
    "K": lambda x: O.rmsnorm_quantize(x[:, :24]),
    "K mx": lambda x: O.rmsnorm_quantize(x[:, :48], had_block=16, fmt="mxfp8"),
    "weight dtype": lambda x: O.rmsnorm_quantize(x, torch.ones(K, dtype=torch.bfloat16)),
    "weight short": lambda x: O.rmsnorm_quantize(x, torch.ones(K - 1)),
    "residual shape": lambda x: O.rmsnorm_quantize(x, None, x[:4]),
    "sum without residual": lambda x: O.rmsnorm_quantize(x, sum_out=x.clone()),
    "sum dtype": lambda x: O.rmsnorm_quantize(x, None, x, sum_out=torch.zeros(M, K)),
    "out short": lambda x: O.rmsnorm_quantize(x, out=i8(M - 1)),
    "out fmt": lambda x: O.rmsnorm_quantize(x, fmt="mxfp8", out=mx(M, K, "mxfp4")),
    "gemv w short": lambda x: O.qgemv_w4a16(bf(), nv(N, K // 2)),
    "gemv a stride": lambda x: O.qgemv_w4a16(O.BF16Tensor(bf(K, M).q.t()), nv(N, K)),
    "gemv bias": lambda x: O.qgemv_w4a8(i8(), nv(N, K), torch.zeros(N + 1)),
    "gemv scales": lambda x: O.qgemv_w4a8(O.INT8Tensor(i8().q, torch.zeros(M - 1)), nv(N, K)),
    "gemv weights mxfp8": lambda x: O.qgemv_mx(mx(M, K), mx(N, K, "mxfp8")),
    "gemv y": lambda x: O.qgemv_mx(mx(M, K), mx(N, K), y=torch.zeros((M, N))),
    "offsets dtype": lambda x: O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), OFF.long()),
    "offsets 2-D": lambda x: O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), OFF[None]),
    "offsets empty": lambda x: O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), OFF[:0]),
    "experts": lambda x: O.qgemm_mx_grouped(mx(M, K), mx(2 * N + 1, K), OFF),
    "grouped bias": lambda x: O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), OFF, torch.zeros(N)),
    "grouped y": lambda x: O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), OFF, y=torch.zeros((M, 2 * N))),
}


@pytest.mark.parametrize("what", list(BAD))
def test_binding_refuses(stub, what):  # noqa: F811
    with pytest.raises(ValueError):
        BAD[what](torch.zeros((M, K), dtype=torch.bfloat16))
    assert stub.calls == []
