"""qgemv_* and qgemm_mx_grouped refuse an output that shares memory with an
operand (workgroups store their columns of Y while others still read all of
A), and accept one whose rows lie around or beside them."""
import ctypes

import pytest
import torch

import video_diffusion_transformer_block_amd as V
from video_diffusion_transformer_block_amd import _lib as L
from helpers import need_gpu

M, N, K, E = 8, 256, 256, 2
MX = dict(aq=(0x1000000, M * K), as_=(0x2000000, M * K // 32), wq=(0x3000000, E * N * K // 2),
          ws=(0x4000000, E * N * K // 32), bias=(0x5000000, 4 * E * N), off=(0x6000000, 4 * (E + 1)))
NV16 = dict(aq=(0x1000000, 2 * M * K), wq=(0x3000000, N * K // 2), ws=(0x4000000, N * K // 16), wts=(0x6000000, 8),
            bias=(0x5000000, 4 * N))
NV8 = dict(NV16, aq=(0x1000000, M * K), as_=(0x2000000, 4 * M))


def call(fn, y, ldy, od):
    b = {"w4a16": NV16, "w4a8": NV8}.get(fn, MX)
    p = {k: ctypes.c_void_p(v[0]) for k, v in b.items()}
    tail = (p["bias"], ctypes.c_void_p(y), ldy, od, M, N, K, None)
    if fn == "w4a16":
        return V.lib().qgemv_w4a16(p["aq"], p["wq"], p["ws"], p["wts"], *tail)
    if fn == "w4a8":
        return V.lib().qgemv_w4a8(p["aq"], p["as_"], p["wq"], p["ws"], p["wts"], *tail)
    if fn == "mx":
        return V.lib().qgemv_mx(L.FMT_MXFP8, p["aq"], p["as_"], p["wq"], p["ws"], *tail)
    return V.lib().qgemm_mx_grouped(L.FMT_MXFP8, p["aq"], p["as_"], p["wq"], p["ws"], p["bias"], p["off"], E,
                                    ctypes.c_void_p(y), ldy, od, M, N, K, None)


def operands(fn):
    b = {"w4a16": NV16, "w4a8": NV8}.get(fn, MX)
    # one expert's weights where the call takes one
    cut = {"wq": 2, "ws": 2, "bias": 2} if fn == "mx" else {}
    return [(k, at, n // cut.get(k, 1)) for k, (at, n) in b.items() if not (fn == "mx" and k == "off")]


@pytest.mark.parametrize("fn", ["w4a16", "w4a8", "mx", "grouped"])
@pytest.mark.parametrize("od", [L.OUT_BF16, L.OUT_F32])
def test_an_output_over_an_operand_is_refused(fn, od):
    es = 4 if od == L.OUT_F32 else 2
    for name, at, n in operands(fn):
        for ldy in (N, N + 64):
            extent = ((M - 1) * ldy + N) * es
            # the same start; the operand's last byte under the first of y; y's last under its first
            for y in (at, at + (n - 1) // es * es, at - extent + es):
                assert call(fn, y, ldy, od) == L.EINVAL, (name, ldy, hex(y))
                assert b"overlaps" in V.lib().vdtq_last_error()
        # right behind y's first row, and longer than the gap to the second
        assert call(fn, at - N * es, N + (n - 1) // es, od) == L.EINVAL and b"overlaps" in V.lib().vdtq_last_error(), name


def test_the_binding_refuses_an_activation_as_output():
    """Square products in place, through the C entry the binding calls."""
    b = torch.zeros((M, K), dtype=torch.bfloat16)
    w, s, ts = torch.zeros((K, K // 2), dtype=torch.uint8), torch.zeros((K, K // 16), dtype=torch.uint8), torch.zeros(2)
    rc = V.lib().qgemv_w4a16(b.data_ptr(), w.data_ptr(), s.data_ptr(), ts.data_ptr(), None, b.data_ptr(), K, L.OUT_BF16,
                             M, K, K, None)
    assert rc == L.EINVAL and b"overlaps" in V.lib().vdtq_last_error()


@pytest.mark.gpu
def test_outputs_between_and_beside_operands():
    """A bias in the columns behind y's, and y right behind the activations:
    the bits of a separate output; an activation as output is refused."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(3)
    k = 256
    x = torch.randn(6, k, device="cuda", generator=g).bfloat16()
    w = V.hadamard_quantize(torch.randn(k, k, device="cuda", generator=g).bfloat16(), 64, "nvfp4")
    bias = torch.randn(k, device="cuda", generator=g)
    a = V.BF16Tensor(x)
    want = V.qgemv_w4a16(a, w, bias, "f32")
    wide = torch.zeros(6, 2 * k, device="cuda")
    wide[2, k:] = bias
    assert torch.equal(V.qgemv_w4a16(a, w, wide[2, k:], "f32", y=wide[:, :k]), want)
    assert torch.equal(wide[2, k:], bias) and (wide[3:, k:] == 0).all()
    both = torch.zeros(12, k, dtype=torch.bfloat16, device="cuda")
    both[:6] = x
    assert torch.equal(V.qgemv_w4a16(V.BF16Tensor(both[:6]), w, bias, y=both[6:]), V.qgemv_w4a16(a, w, bias))
    assert torch.equal(both[:6], x)
    for y in (both[:6], both[3:9]):
        with pytest.raises(V.VdtqError, match="overlaps"):
            V.qgemv_w4a16(V.BF16Tensor(both[:6]), w, bias, y=y)
    assert torch.equal(both[:6], x)
