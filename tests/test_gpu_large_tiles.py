"""The 256 x 256 tiles of qgemm_mx_grouped at sizes that choose them: K of few
stages, with and without scale quads, outputs of any stride, and a captured
call replayed with other row counts.  (bf16 output of both formats and fp32
output of MXFP4 rows; fp32 output of MXFP8 rows takes the exact 64 x 128
tiles.)"""
import numpy as np
import pytest
import torch

import video_diffusion_transformer_block_amd as V
from helpers import log, need_gpu
from test_gpu_few_rows import dev
from test_gpu_many_experts import exact_and_cut

pytestmark = pytest.mark.gpu
N = 3400            # 4096 rows: 14 feature tiles x 16 row tiles, one round of the card


def operands(T, E, K, afmt, n=N):
    g = torch.Generator(device="cuda").manual_seed(T + K)
    return (V.hadamard_quantize(torch.randn(T, K, device="cuda", generator=g).bfloat16(), 64, afmt),
            V.hadamard_quantize(torch.randn(E * n, K, device="cuda", generator=g).bfloat16(), 64, "mxfp4"),
            torch.randn(E, n, device="cuda", generator=g))


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("K", [128, 256, 384, 512, 640])
def test_few_stages(afmt, K):
    need_gpu()
    log(f"large tiles {afmt} K={K}")
    a, w, b = operands(4096, 1, K, afmt)
    off = np.array([0, 4096], np.int32)
    want, terms, cut = exact_and_cut(a, w, off, afmt, N)
    want, terms = want + b.double(), terms + b.double().abs()
    bound = 2 * (K + 4) * 2.0 ** -24 * terms             # as in test_gpu_many_experts
    for od in ("bf16", "f32"):
        y = V.qgemm_mx_grouped(a, w, dev(off), b, od).double()
        torch.cuda.synchronize()
        tol = bound if od == "f32" else bound + cut + 2.0 ** -8 * (want.abs() + bound + cut)
        assert ((y - want).abs() <= tol).all()


@pytest.mark.parametrize("afmt", ["mxfp8", "mxfp4"])
def test_output_strides(afmt):
    need_gpu()
    T, E, K = 4096, 2, 256
    a, w, b = operands(T, E, K, afmt)
    off = dev(np.array([3, 2050, T - 5], np.int32))
    for od, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        want = V.qgemm_mx_grouped(a, w, off, b, od, y=torch.full((T, N), 7.0, dtype=dt, device="cuda"))
        for pad, shift in ((8, 0), (8, 8), (5, 3)):
            log(f"strides {afmt} {od} pad={pad} shift={shift}")
            wide = torch.full((T + 1, N + pad), 7.0, dtype=dt, device="cuda")
            y = V.qgemm_mx_grouped(a, w, off, b, od, y=wide[:T, shift:N + shift])
            torch.cuda.synchronize()
            assert torch.equal(y, want)
            wide[3:T - 5, shift:N + shift] = 7.0
            assert (wide == 7.0).all()


@pytest.mark.parametrize("T,E,n", [(4096, 3, N), (300, 4, 136)])
def test_replays_with_other_row_counts(T, E, n):
    """Large tiles, and small ones: captured calls replayed after the offsets
    and the rows changed, with eager calls in between."""
    need_gpu()
    K = 256
    rng = np.random.Generator(np.random.PCG64(T))
    counts = [np.sort(rng.integers(0, T + 1, size=E + 1)) for _ in range(3)] + [np.array([0] * E + [T]), np.full(E + 1, T)]
    off = dev(np.linspace(0, T, E + 1).astype(np.int32))
    a8, w, b = operands(T, E, K, "mxfp8", n)
    a4, _, _ = operands(T, E, K, "mxfp4", n)
    ins = [(a8, "bf16"), (a8, "f32"), (a4, "bf16"), (a4, "f32")]

    def calls(ys):
        return [V.qgemm_mx_grouped(a, w, off, b, od, y=y) for (a, od), y in zip(ins, ys)]

    def fresh():
        return [torch.full((T, n), 7.0, dtype=torch.bfloat16 if od == "bf16" else torch.float32, device="cuda")
                for _, od in ins]

    ys = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(ys)
    for k, c in enumerate(counts):
        log(f"replay {k} T={T} offsets {c.tolist()}")
        off.copy_(dev(c.astype(np.int32)))
        a8.q.copy_(a8.q.roll(1, 0))
        for y in ys:
            y.fill_(7.0)
        graph.replay()
        want = calls(fresh())
        torch.cuda.synchronize()
        assert all(torch.equal(y, v) for y, v in zip(ys, want))
        assert all((y[:c[0]] == 7.0).all() and (y[c[-1]:] == 7.0).all() for y in ys)
