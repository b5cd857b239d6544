"""The products with few rows (up to 16 a group, B stored N×K, csrc/gemm_rows.hpp): four waves take a
row's chunks of 256 bytes in turn, two sets of registers alternating, and the chunk that is not whole
falls to the wave whose turn it is.  The lengths here give every wave that last chunk, rows without a
whole chunk, and up to nine rounds of whole ones.

Operands are small integers (16 bits: |sum| <= 16·K) or codes with scale 1 (4 bits: multiples of 1/4 of
at most 36, |sum| <= 144·K quarters), below 2^24 for every K here, so fp32 holds every sum and the
output must equal the reference rounded once, whatever the order."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from tests.test_grouped import _dev, _gen, _ints, _offsets, _ref_rows
from tests.test_mx4 import _random_mx4

gpu = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# rows of each group, and rows before the first and behind the last; one group of more than 16 rows
# takes two workgroup tiles
SIZES = [([1], 0, 0), ([2], 0, 0), ([16], 0, 0), ([0, 1, 0, 16, 3], 1, 2), ([1, 0, 30, 2, 0, 5], 1, 2)]
# 16 bits: whole chunks of 128 values and values left: 0+40, 1+8, 2+16, 3+24, 4+0, 8+8, 9+8, 16+8, 32+8, 35+100
K16 = [40, 136, 272, 408, 512, 1032, 1160, 2056, 4104, 4580]
# 4 bits, chunks of 512 values: 0+96, 1+32, 2+64, 3+480, 4+32, 8+0, 9+32, 12+256, 16+0
K4 = [96, 544, 1088, 2016, 2080, 4096, 4640, 6400, 8192]


def _ops():
    from tiled_bf16_gemm_amd import torch_ops
    return torch_ops


def _edges(case):
    """Group borders, all rows, and the rows that belong to a group."""
    sizes, before, behind = case
    edges = _offsets(sizes, before)
    return edges, edges[-1] + behind, slice(before, edges[-1])


def _operands16(case, N, K, dtype, seed):
    gen, (edges, M, inside) = _gen(seed), _edges(case)
    A = _ints(gen, (M, K), TORCH[dtype])
    B = _ints(gen, (len(case[0]), N, K), TORCH[dtype])
    want = _ref_rows(A, B, edges, "nk")
    A[:inside.start], A[inside.stop:] = float("nan"), float("nan")
    for e, n in enumerate(case[0]):
        if n == 0:
            B[e] = float("nan")
    return A, B, edges, inside, want


def _operands4(case, N, K):
    rng, (edges, M, inside) = np.random.default_rng(K), _edges(case)
    a, sa, va = _random_mx4(rng, (M,), K, spread=0)
    b, sb, vb = _random_mx4(rng, (len(case[0]), N), K, spread=0)
    sa[:inside.start], sa[inside.stop:] = 255, 255
    for e, n in enumerate(case[0]):
        if n == 0:
            sb[e] = 255
    return a, sa, va, b, sb, vb, edges, inside


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", K16)
@pytest.mark.parametrize("case", SIZES)
def test_rows_exact(case, K, dtype):
    N = 83
    print(f"few rows {dtype} {case} K={K}", flush=True)
    A, B, edges, inside, want = _operands16(case, N, K, dtype, K)
    for out_dtype in ("f32", dtype):
        out = torch.full((A.shape[0], N), -77.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().gemm_grouped(A, B, _dev(edges), "nk", out_dtype, out=out)
        assert torch.equal(out[inside], want[inside].to(out.dtype)), out_dtype
        assert (out[:inside.start] == -77).all() and (out[inside.stop:] == -77).all()


@gpu
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("K", [1160, 0])
def test_rows_alpha_beta(K, dtype, out_dtype):
    """Powers of two: exact, then rounded once.  beta == 0 must not read C, alpha == 0 neither A nor B."""
    N = 75
    A, B, edges, inside, S = _operands16(SIZES[3], N, K, dtype, 3)
    C = _ints(_gen(4), (A.shape[0], N), TORCH[out_dtype])
    for alpha, beta in ((0.5, 0.0), (1.0, 1.0), (-2.0, 0.25), (0.0, 2.0), (0.0, 0.0)):
        out = C.clone()
        if beta == 0.0:
            out[inside] = float("nan")
        keep = out.clone()
        a = torch.full_like(A, float("nan")) if alpha == 0.0 else A
        _ops().gemm_grouped(a, B, _dev(edges), "nk", out_dtype, out=out, alpha=alpha, beta=beta)
        want = alpha * S + (beta * C.double() if beta else 0.0)
        assert torch.equal(out[inside], want[inside].to(out.dtype)), (alpha, beta)
        for rest in (slice(0, inside.start), slice(inside.stop, None)):
            assert torch.equal(out[rest].view(torch.uint8), keep[rest].view(torch.uint8))


@gpu
@pytest.mark.parametrize("K", K4)
@pytest.mark.parametrize("case", SIZES)
def test_mx4_exact(case, K):
    """Ragged, and dense where there is one group; scale 1."""
    N, G = 83, len(case[0])
    print(f"few rows mx4 {case} K={K}", flush=True)
    a, sa, va, b, sb, vb, edges, inside = _operands4(case, N, K)
    want = torch.full((a.shape[0], N), -9.0, dtype=torch.float64, device="cuda")
    for e in range(G):
        rows = slice(edges[e], edges[e + 1])
        want[rows] = va[rows] @ vb[e].t().contiguous()
    for out_dtype in ("f32", "bf16"):
        out = torch.full(want.shape, -9.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().mx4_gemm_grouped(a, sa, b, sb, _dev(edges), out_dtype, out=out)
        assert torch.equal(out, want.to(out.dtype)), out_dtype
        if G == 1:
            assert torch.equal(_ops().mx4_gemm(a, sa, b[0], sb[0], out_dtype), want.to(out.dtype)), out_dtype


def _child():
    """One call of each kind and size above, for the log; prints their number."""
    ops, calls = _ops(), 0
    for case in SIZES:
        for K in K16:
            for dtype in ("bf16", "f16"):
                A, B, edges, _, _ = _operands16(case, 83, K, dtype, K)
                ops.gemm_grouped(A, B, _dev(edges), "nk", dtype)
                calls += 1
        for K in K4:
            a, sa, _, b, sb, _, edges, _ = _operands4(case, 83, K)
            ops.mx4_gemm_grouped(a, sa, b, sb, _dev(edges))
            calls += 1
            if len(case[0]) == 1:
                ops.mx4_gemm(a, sa, b[0], sb[0])
                calls += 1
    torch.cuda.synchronize()
    print(f"{calls} calls", flush=True)


@gpu
def test_these_sizes_take_the_kernel_of_few_rows():
    r = subprocess.run([sys.executable, "-m", "tests.test_few_rows"], capture_output=True, text=True, timeout=100,
                       cwd=ROOT, env=dict(os.environ, TBG_LOG="1"))
    assert r.returncode == 0, r.stderr[-3000:]
    lines = [t for t in r.stderr.splitlines() if "gemm groups=" in t]
    assert f"{len(lines)} calls" in r.stdout
    assert all("rows 16x16" in t for t in lines), [t for t in lines if "rows 16x16" not in t][:3]


if __name__ == "__main__":
    _child()
