"""What a call makes of the library's status when it comes through the native
marshalling module: a refusal (VDTQ_EINVAL, VDTQ_EUNSUPPORTED) goes to the
Python path, which names it; any other failure is raised at once, never
answered by making the call a second time.  And a call's status is its own:
an error that other code left pending on the thread is neither reported by
the call nor makes it run twice."""
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from video_diffusion_transformer_block_amd import _lib as L
from video_diffusion_transformer_block_amd import ops as O
from helpers import need_gpu
from test_ops_validation import mx, nv, stub  # noqa: F401

M, N, K = 8, 64, 128


class _Native:
    """Every entry answers with the given status and counts its calls."""

    def __init__(self, rc):
        self.rc, self.calls = rc, 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return self.rc
        return call


CALLS = {
    "norm": lambda: O.rmsnorm_quantize(torch.zeros((M, K), dtype=torch.bfloat16)),
    "w4a16": lambda: O.qgemv_w4a16(O.BF16Tensor(torch.zeros((M, K), dtype=torch.bfloat16)), nv(N, K)),
    "w4a8": lambda: O.qgemv_w4a8(O.INT8Tensor(torch.zeros((M, K), dtype=torch.int8), torch.zeros(M)), nv(N, K)),
    "mx": lambda: O.qgemv_mx(mx(M, K, "mxfp8"), mx(N, K)),
    "grouped": lambda: O.qgemm_mx_grouped(mx(M, K), mx(2 * N, K), torch.zeros(3, dtype=torch.int32)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_a_failed_native_call_is_raised_and_not_repeated(stub, monkeypatch, name):  # noqa: F811
    native = _Native(L.EHIP)
    monkeypatch.setattr(O, "_fast", native)
    monkeypatch.setattr(stub, "vdtq_last_error", lambda: b"launch", raising=False)
    with pytest.raises(V.VdtqError) as e:
        CALLS[name]()
    assert e.value.code == L.EHIP
    assert native.calls == 1 and stub.calls == []


@pytest.mark.parametrize("name", list(CALLS))
def test_a_declined_native_call_takes_the_python_path(stub, monkeypatch, name):  # noqa: F811
    native = _Native(None)
    monkeypatch.setattr(O, "_fast", native)
    CALLS[name]()
    assert native.calls == 1 and len(stub.calls) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("native", [True, False])
def test_a_pending_error_of_other_code_does_not_touch_the_calls(monkeypatch, native):
    need_gpu()
    assert O._fast is not None, "the native entry is not built"
    if not native:
        monkeypatch.setattr(O, "_fast", None)
    g = torch.Generator(device="cuda").manual_seed(9)

    def rand(rows):
        return torch.randn(rows, 512, device="cuda", generator=g).bfloat16()

    x, res, many = rand(40), rand(40), rand(2000)
    w, wide = (V.hadamard_quantize(rand(n), 64, "mxfp4") for n in (192, 7168))
    wn = V.hadamard_quantize(rand(192), 64, "nvfp4")
    off = torch.tensor([0, 20, 20, 40], dtype=torch.int32, device="cuda")
    one = torch.tensor([0, 2000], dtype=torch.int32, device="cuda")

    def calls(pending):
        x1, x2 = x.clone(), x.clone()
        if pending:
            # a device that does not exist: the runtime refuses it, changes
            # nothing, and keeps the error as the thread's last one
            assert V.lib().hipSetDevice(1 << 20) != 0
        a8, s1 = V.rmsnorm_quantize(x1, None, res, fmt="int8", sum_out=x1)
        amx, s2 = V.rmsnorm_quantize(x2, None, res, fmt="mxfp8", sum_out=x2)
        a16, _ = V.rmsnorm_quantize(x2, fmt="bf16")
        rmx, _ = V.rmsnorm_quantize(many, fmt="mxfp8")
        out = [s1, s2, a8.q, a8.scales, amx.q, a16.q, V.qgemv_w4a8(V.INT8Tensor(a8.q[:7], a8.scales[:7]), wn),
               V.qgemv_w4a16(V.BF16Tensor(a16.q[:7]), wn), V.qgemv_mx(V.MXTensor(amx.q[:7], amx.scales[:7], "mxfp8"), w)]
        # rows by expert: few-row kernels or small tiles, and large tiles
        for od in ("bf16", "f32"):
            out += [V.qgemm_mx_grouped(amx, w, off, None, od), V.qgemm_mx_grouped(rmx, wide, one, None, od)]
        left = V.lib().hipGetLastError()                # ours, taken back
        torch.cuda.synchronize()
        return [t.cpu() for t in out], left

    # (the second run finds the first one's memory in torch's cache: torch
    # itself raises pending errors where it asks the runtime for more)
    want, _ = calls(False)
    got, left = calls(True)
    assert torch.equal(got[0], (x.float() + res.float()).bfloat16().cpu())      # the addition, once
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert left != 0                                    # and still there for whoever caused it
