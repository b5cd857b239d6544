"""Products over ragged groups (tbg_gemm_grouped, tbg_gemm_grouped_wgrad) against the same products in
64 bits.

Operands of small integers have sums that fp32 holds exactly (|sum| <= 16·K < 2^24), so there the
output must equal the reference rounded once to C's type, bit for bit, whatever the order of the sum.
Real operands are held to the bound of an fp32 sum of K exact products, each addition off by at
most one unit in the last place (2^-23 relative to the sum of magnitudes so far), plus the half step
of rounding to C's type: |C - exact| <= K·2^-23·sum|a·b| + eps/2·(|exact| + that)."""
import numpy as np
import pytest
import torch

import tiled_bf16_gemm_amd as tbg

gpu = pytest.mark.gpu
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PTR = 0x7F00_0000_0000  # a device-like address: argument checks never touch memory


def _ops():
    from tiled_bf16_gemm_amd import torch_ops
    return torch_ops


def _ints(gen, shape, dtype):
    return torch.randint(-4, 5, shape, generator=gen, device="cuda").to(dtype)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _offsets(sizes, first=0):
    return [first] + [first + int(v) for v in np.cumsum(sizes)]


def _dev(edges):
    return torch.tensor(edges, dtype=torch.int32, device="cuda")


def _padded(t, ld, fill=float("nan")):
    """The same matrix (or stack) with rows ld elements apart, NaN in between."""
    full = torch.full((*t.shape[:-1], ld), fill, dtype=t.dtype, device=t.device)
    full[..., :t.shape[-1]] = t
    return full[..., :t.shape[-1]]


def _ref_rows(A, B, edges, layout):
    out = torch.zeros((A.shape[0], B.shape[2] if layout == "kn" else B.shape[1]), dtype=torch.float64, device=A.device)
    for e in range(len(edges) - 1):
        lo, hi = edges[e], edges[e + 1]
        b = B[e].double()
        out[lo:hi] = A[lo:hi].double() @ (b if layout == "kn" else b.t().contiguous())
    return out


def _ref_wgrad(X, Y, edges):
    return torch.stack([X[lo:hi].double().t().contiguous() @ Y[lo:hi].double() for lo, hi in zip(edges, edges[1:])])


def _bound(exact, magnitude, terms, dtype):
    acc = terms * 2.0 ** -23 * magnitude
    return acc + torch.finfo(dtype).eps / 2 * (exact.abs() + acc)


# ---- refusals (CPU) -------------------------------------------------------------------------------

def _rows_args(**over):
    a = dict(groups=2, M=8, N=16, K=24, offsets=PTR, alpha=1.0, A=PTR, lda=24, B=PTR, ldb=16, stride_b=24 * 16,
             b_layout="kn", ab_dtype="bf16", beta=0.0, C=PTR, ldc=16, c_dtype="f32")
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(groups=-1), tbg.ERR_INVALID_VALUE),
    (dict(M=-1), tbg.ERR_INVALID_VALUE),
    (dict(N=-1), tbg.ERR_INVALID_VALUE),
    (dict(K=-1), tbg.ERR_INVALID_VALUE),
    (dict(groups=4097), tbg.ERR_UNSUPPORTED),
    (dict(M=(1 << 30) + 1), tbg.ERR_UNSUPPORTED),
    (dict(offsets=0), tbg.ERR_INVALID_VALUE),
    (dict(offsets=PTR + 2), tbg.ERR_MISALIGNED),
    (dict(A=0), tbg.ERR_INVALID_VALUE),
    (dict(B=0), tbg.ERR_INVALID_VALUE),
    (dict(C=0), tbg.ERR_INVALID_VALUE),
    (dict(lda=23), tbg.ERR_INVALID_VALUE),
    (dict(lda=1 << 22), tbg.ERR_UNSUPPORTED),
    (dict(ldb=15), tbg.ERR_INVALID_VALUE),
    (dict(ldc=15), tbg.ERR_INVALID_VALUE),
    (dict(stride_b=24 * 16 - 1), tbg.ERR_INVALID_VALUE),
    (dict(stride_b=0), tbg.ERR_INVALID_VALUE),
    (dict(b_layout=2), tbg.ERR_INVALID_VALUE),
    (dict(ab_dtype="f32"), tbg.ERR_INVALID_VALUE),
    (dict(ab_dtype="f8e4m3"), tbg.ERR_INVALID_VALUE),
    (dict(c_dtype="f16"), tbg.ERR_INVALID_VALUE),
    (dict(ab_dtype="f16", c_dtype="bf16"), tbg.ERR_INVALID_VALUE),
    (dict(lda=25), tbg.ERR_OUT_OF_RANGE),                           # a repack without a workspace
    (dict(lda=25, workspace=PTR + 64, workspace_bytes=1 << 20), tbg.ERR_MISALIGNED),
])
def test_rows_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.gemm_grouped(**_rows_args(**over))
    assert e.value.status == status, e.value


def _wgrad_args(**over):
    a = dict(groups=2, M=8, P=16, Q=24, offsets=PTR, alpha=1.0, X=PTR, ldx=16, Y=PTR, ldy=24, ab_dtype="bf16", beta=0.0,
             C=PTR, ldc=24, stride_c=16 * 24, c_dtype="f32")
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(groups=-1), tbg.ERR_INVALID_VALUE),
    (dict(P=-1), tbg.ERR_INVALID_VALUE),
    (dict(groups=4097), tbg.ERR_UNSUPPORTED),
    (dict(Q=(1 << 30) + 1, ldy=1 << 31, ldc=1 << 31), tbg.ERR_UNSUPPORTED),
    (dict(offsets=0), tbg.ERR_INVALID_VALUE),
    (dict(X=0), tbg.ERR_INVALID_VALUE),
    (dict(Y=0), tbg.ERR_INVALID_VALUE),
    (dict(C=0), tbg.ERR_INVALID_VALUE),
    (dict(ldx=15), tbg.ERR_INVALID_VALUE),
    (dict(ldy=23), tbg.ERR_INVALID_VALUE),
    (dict(ldc=23), tbg.ERR_INVALID_VALUE),
    (dict(stride_c=16 * 24 - 1), tbg.ERR_INVALID_VALUE),
    (dict(c_dtype="f16"), tbg.ERR_INVALID_VALUE),
    (dict(ab_dtype="f8e5m2"), tbg.ERR_INVALID_VALUE),
    (dict(X=PTR + 2), tbg.ERR_OUT_OF_RANGE),
])
def test_wgrad_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.gemm_grouped_wgrad(**_wgrad_args(**over))
    assert e.value.status == status, e.value


def test_empty_calls_need_no_device():
    tbg.gemm_grouped(**_rows_args(groups=0, offsets=0))
    tbg.gemm_grouped(**_rows_args(M=0, A=0, C=0))
    tbg.gemm_grouped(**_rows_args(N=0, ldb=1, ldc=1, stride_b=0, B=0, C=0))
    tbg.gemm_grouped_wgrad(**_wgrad_args(groups=0, offsets=0))
    tbg.gemm_grouped_wgrad(**_wgrad_args(P=0, ldx=1, stride_c=0, C=0))


def test_workspace_queries():
    q = tbg.gemm_grouped_workspace_query
    assert q(2, 8, 16, 24, "bf16", PTR, 24, PTR, 16, 24 * 16, "kn") == 0
    assert q(2, 8, 16, 24, "bf16", PTR, 25, PTR, 16, 24 * 16, "kn") == 512                # 8·24·2 -> 512
    assert q(2, 8, 16, 24, "bf16", PTR + 2, 24, PTR, 16, 24 * 16, "kn") == 512
    assert q(2, 8, 16, 21, "bf16", PTR, 24, PTR, 24, 24 * 16, "nk") == 512 + 2 * 16 * 24 * 2
    assert q(2, 8, 16, 24, "bf16", PTR, 24, PTR, 16, 24 * 16 + 4, "kn") == 2 * 24 * 16 * 2  # second matrix off 16 bytes
    assert q(1, 8, 16, 24, "bf16", PTR, 24, PTR, 16, 24 * 16 + 4, "kn") == 0
    assert q(2, 8, 16, 24, "f8e4m3", PTR, 25, PTR, 16, 24 * 16, "kn") == 0
    w = tbg.gemm_grouped_wgrad_workspace_query
    assert w(2, 8, 16, 24, "f16", PTR, 16, PTR, 24) == 0
    assert w(2, 8, 13, 24, "f16", PTR, 13, PTR, 24) == 256
    assert w(2, 8, 13, 24, "f16", PTR, 16, PTR + 8, 24) == 512


# ---- the rows' product ----------------------------------------------------------------------------

# (group sizes, rows before the first, rows behind the last, N, K): one token, odd sizes, tiles that
# overhang, groups without a row, many groups, sizes that take each tile
CASES = [
    ([1], 0, 0, 1, 1),
    ([1], 0, 0, 16, 8),
    ([0, 0, 0], 0, 5, 24, 40),
    ([3, 0, 1, 0, 7], 0, 4, 40, 72),
    ([5, 64, 0, 65, 1], 2, 3, 130, 100),
    ([33, 31], 0, 0, 67, 129),
    ([1] * 70 + [0] * 3 + [9], 0, 1, 64, 64),
    ([2] * 200, 0, 0, 96, 200),
    ([130, 0, 257, 700], 0, 9, 520, 192),
    ([700, 1200, 0, 133], 1, 0, 1030, 328),
    ([2100, 1900], 0, 17, 4100, 72),
]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rows_exact(case, layout, dtype):
    sizes, before, behind, N, K = CASES[case]
    edges = _offsets(sizes, before)
    M, G, dt = edges[-1] + behind, len(sizes), TORCH[dtype]
    print(f"rows {dtype} {layout} groups={G} M={M} N={N} K={K}", flush=True)
    gen = _gen(case)
    A = _ints(gen, (M, K), dt)
    B = _ints(gen, (G, K, N) if layout == "kn" else (G, N, K), dt)
    want = _ref_rows(A, B, edges, layout)
    # what must not be looked at: rows of no group, matrices of groups without rows
    A[:before], A[edges[-1]:] = float("nan"), float("nan")
    for e, n in enumerate(sizes):
        if n == 0:
            B[e] = float("nan")
    for out_dtype in ("f32", dtype):
        out = torch.full((M, N), -77.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().gemm_grouped(A, B, _dev(edges), layout, out_dtype, out=out)
        assert torch.equal(out[before:edges[-1]], want[before:edges[-1]].to(out.dtype)), out_dtype
        assert (out[:before] == -77).all() and (out[edges[-1]:] == -77).all()


@gpu
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_real_operands(dtype, layout):
    edges, N, K = _offsets([300, 0, 17, 451], 3), 264, 1000
    dt, gen = TORCH[dtype], _gen(5)
    A = torch.randn((edges[-1], K), generator=gen, device="cuda").to(dt)
    B = (torch.randn((4, K, N) if layout == "kn" else (4, N, K), generator=gen, device="cuda") * 0.05).to(dt)
    want, mag = _ref_rows(A, B, edges, layout), _ref_rows(A.abs(), B.abs(), edges, layout)
    for out_dtype in ("f32", dtype):
        out = _ops().gemm_grouped(A, B, _dev(edges), layout, out_dtype)
        err = (out.double() - want).abs()[3:]
        assert (err <= _bound(want, mag, K, out.dtype)[3:]).all(), err.max().item()


@gpu
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("where", ["pitch", "odd_pitch", "odd_base", "odd_stride", "strided_odd"])
def test_rows_strides_and_alignment(where, layout):
    """Pitched operands with NaN between the rows and the matrices, and every reason for a repack."""
    edges, N, K, G = _offsets([40, 0, 90], 0), 72, 88, 3
    gen, dt = _gen(9), torch.bfloat16
    A, B = _ints(gen, (130, K), dt), _ints(gen, (G, K, N) if layout == "kn" else (G, N, K), dt)
    want = _ref_rows(A, B, edges, layout)
    cols, rows = B.shape[2], B.shape[1]
    if where == "pitch":
        A, B = _padded(A, K + 8), _padded(B, cols + 16)
    elif where == "odd_pitch":
        A, B = _padded(A, K + 3), _padded(B, cols + 5)
    elif where == "odd_base":
        flat = torch.full((130 * K + 1,), float("nan"), dtype=dt, device="cuda")
        flat[1:] = A.reshape(-1)
        A = flat[1:].view(130, K)
        flat = torch.full((G * rows * cols + 3,), float("nan"), dtype=dt, device="cuda")
        flat[3:] = B.reshape(-1)
        B = flat[3:].view(G, rows, cols)
    else:
        # one matrix in every (rows + 1) · ld elements, ld odd or even
        ld = cols + (3 if where == "strided_odd" else 8)
        full = torch.full((G, rows + 1, ld), float("nan"), dtype=dt, device="cuda")
        full[:, :rows, :cols] = B
        B = full[:, :rows, :cols]
        if where == "odd_stride":  # matrices an odd number of elements apart
            flat = torch.full((G * (rows * cols + 5),), float("nan"), dtype=dt, device="cuda")
            odd = flat.as_strided((G, rows, cols), (rows * cols + 5, cols, 1))
            odd.copy_(B)
            B = odd
    for N_out in (N + 1, N + 8):
        full = torch.full((130, N_out), -7.0, dtype=dt, device="cuda")
        _ops().gemm_grouped(A, B, _dev(edges), layout, "bf16", out=full[:, :N])
        assert torch.equal(full[:, :N], want.to(dt))
        assert (full[:, N:] == -7).all()


@gpu
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f16", "f32")])
def test_rows_alpha_beta(dtype, out_dtype):
    """alpha·S + beta·C in fp32 with powers of two: exact, then rounded once.  beta == 0 must not read C,
    alpha == 0 neither A nor B; K == 0 is the empty sum."""
    edges, N, K, dt = _offsets([20, 0, 111], 2), 75, 64, TORCH[dtype]
    M, gen = edges[-1] + 3, _gen(11)
    A, B, C = _ints(gen, (M, K), dt), _ints(gen, (3, K, N), dt), _ints(gen, (M, N), TORCH[out_dtype])
    S = _ref_rows(A, B, edges, "kn")
    inside = slice(edges[0], edges[-1])
    for alpha, beta in ((0.5, 0.0), (1.0, 1.0), (-2.0, 0.25), (0.0, 2.0), (0.0, 0.0)):
        out = C.clone()
        if beta == 0.0:
            out[inside] = float("nan")
        keep = out.clone()
        a = torch.full_like(A, float("nan")) if alpha == 0.0 else A
        _ops().gemm_grouped(a, B, _dev(edges), "kn", out_dtype, out=out, alpha=alpha, beta=beta)
        want = alpha * S + (beta * C.double() if beta else 0.0)
        assert torch.equal(out[inside], want[inside].to(out.dtype)), (alpha, beta)
        assert torch.equal(out[:2].view(torch.uint8), keep[:2].view(torch.uint8))
        assert torch.equal(out[edges[-1]:].view(torch.uint8), keep[edges[-1]:].view(torch.uint8))
    out = torch.full((M, N), 3.0, dtype=TORCH[out_dtype], device="cuda")
    _ops().gemm_grouped(A[:, :0], B[:, :0], _dev(edges), "kn", out_dtype, out=out)
    assert (out[inside] == 0).all() and (out[:2] == 3).all()
    out = torch.full((M, N), 3.0, dtype=TORCH[out_dtype], device="cuda")
    _ops().gemm_grouped(A[:, :0], B[:, :0], _dev(edges), "kn", out_dtype, out=out, beta=2.0)
    assert (out[inside] == 6).all() and (out[edges[-1]:] == 3).all()


# Sizes that take the 256×256 tile (test_grouped_handoff.py checks the choice for the same sizes):
# several tiles a group, overhang on every side, a group without rows and one of one row past a tile.
LARGE_ROWS = ([1200, 0, 800, 257, 1743], 2, 7, 3402, 1276)
LARGE_GRAD = ([1200, 0, 1800, 257, 2743], 1, 2, 2003, 2058)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_rows_exact_on_the_large_tile(layout, dtype):
    sizes, before, behind, N, K = LARGE_ROWS
    edges, G, dt = _offsets(sizes, before), len(sizes), TORCH[dtype]
    M = edges[-1] + behind
    print(f"rows {dtype} {layout} groups={G} M={M} N={N} K={K}", flush=True)
    gen = _gen(70)
    A, B = _ints(gen, (M, K), dt), _ints(gen, (G, K, N) if layout == "kn" else (G, N, K), dt)
    want = _ref_rows(A, B, edges, layout)
    A[:before], A[edges[-1]:], B[1] = float("nan"), float("nan"), float("nan")
    inside = slice(before, edges[-1])
    for out_dtype in ("f32", dtype):
        out = torch.full((M, N), -77.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().gemm_grouped(A, B, _dev(edges), layout, out_dtype, out=out)
        assert torch.equal(out[inside], want[inside].to(out.dtype)), out_dtype
        assert (out[:before] == -77).all() and (out[edges[-1]:] == -77).all()
    out.fill_(2.0)
    _ops().gemm_grouped(A, B, _dev(edges), layout, dtype, out=out, alpha=2.0, beta=-3.0)
    assert torch.equal(out[inside], (2 * want[inside] - 6).to(dt))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wgrad_exact_on_the_large_tile(dtype):
    sizes, before, behind, P, Q = LARGE_GRAD
    edges, G, dt = _offsets(sizes, before), len(sizes), TORCH[dtype]
    M = edges[-1] + behind
    print(f"wgrad {dtype} groups={G} M={M} P={P} Q={Q}", flush=True)
    gen = _gen(71)
    X, Y = _ints(gen, (M, P), dt), _ints(gen, (M, Q), dt)
    want = _ref_wgrad(X, Y, edges)
    for t in (X, Y):
        t[:before], t[edges[-1]:] = float("nan"), float("nan")
    for out_dtype in ("f32", dtype):
        out = torch.full((G, P, Q), float("nan"), dtype=TORCH[out_dtype], device="cuda")
        _ops().gemm_grouped_wgrad(X, Y, _dev(edges), out_dtype, out=out)
        assert torch.equal(out, want.to(out.dtype)), out_dtype
    out.fill_(4.0)
    _ops().gemm_grouped_wgrad(X, Y, _dev(edges), dtype, out=out, alpha=0.5, beta=1.0)
    assert torch.equal(out, (0.5 * want + 4).to(dt))


@gpu
def test_rows_infinities_stay_in_their_group():
    edges, N, K, dt = _offsets([10, 20, 30], 0), 40, 48, torch.bfloat16
    gen = _gen(13)
    A, B = _ints(gen, (60, K), dt), _ints(gen, (3, N, K), dt)
    want = _ref_rows(A, B, edges, "nk").to(dt)
    A[12, 3], B[1, 5, 7] = float("inf"), float("nan")
    out = _ops().gemm_grouped(A, B, _dev(edges), "nk", "bf16")
    assert torch.equal(out[:10], want[:10]) and torch.equal(out[30:], want[30:])
    clean = torch.ones(N, dtype=torch.bool, device="cuda")
    clean[5] = False
    rows = [r for r in range(10, 30) if r != 12]
    assert torch.equal(out[rows][:, clean], want[rows][:, clean])
    assert out[10:30, 5].isnan().all() and not out[12].isfinite().any()


# ---- the weight gradient ---------------------------------------------------------------------------

WGRAD = [
    ([1], 0, 0, 1, 1),
    ([0, 0], 0, 3, 9, 17),
    ([3, 0, 1, 0, 7], 1, 4, 40, 72),
    ([63, 64, 65, 0, 200], 0, 3, 130, 100),
    ([33, 31], 0, 0, 67, 129),
    ([1] * 70 + [0] * 3 + [9], 0, 1, 64, 64),
    ([500, 1, 128], 3, 9, 520, 392),
    ([300, 277], 0, 0, 2056, 2048),
    ([129] * 9, 0, 0, 1032, 1096),
]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("case", range(len(WGRAD)))
def test_wgrad_exact(case, dtype):
    sizes, before, behind, P, Q = WGRAD[case]
    edges = _offsets(sizes, before)
    M, G, dt = edges[-1] + behind, len(sizes), TORCH[dtype]
    print(f"wgrad {dtype} groups={G} M={M} P={P} Q={Q}", flush=True)
    gen = _gen(100 + case)
    X, Y = _ints(gen, (M, P), dt), _ints(gen, (M, Q), dt)
    want = _ref_wgrad(X, Y, edges)
    for t in (X, Y):
        t[:before], t[edges[-1]:] = float("nan"), float("nan")
    for out_dtype in ("f32", dtype):
        out = torch.full((G, P, Q), float("nan"), dtype=TORCH[out_dtype], device="cuda")
        _ops().gemm_grouped_wgrad(X, Y, _dev(edges), out_dtype, out=out)
        assert torch.equal(out, want.to(out.dtype)), out_dtype


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wgrad_real_operands(dtype):
    edges, P, Q, dt = _offsets([300, 0, 1700, 451], 3), 264, 200, TORCH[dtype]
    gen = _gen(6)
    X = torch.randn((edges[-1], P), generator=gen, device="cuda").to(dt)
    Y = (torch.randn((edges[-1], Q), generator=gen, device="cuda") * 0.05).to(dt)
    want, mag = _ref_wgrad(X, Y, edges), _ref_wgrad(X.abs(), Y.abs(), edges)
    for out_dtype in ("f32", dtype):
        out = _ops().gemm_grouped_wgrad(X, Y, _dev(edges), out_dtype)
        err = (out.double() - want).abs()
        assert (err <= _bound(want, mag, 1700, out.dtype)).all(), err.max().item()


@gpu
@pytest.mark.parametrize("pad_x,pad_y,off", [(8, 0, 0), (3, 8, 0), (0, 5, 0), (0, 0, 1), (16, 24, 8)])
def test_wgrad_strides_alignment_and_accumulation(pad_x, pad_y, off):
    edges, P, Q, dt = _offsets([40, 0, 91], 0), 72, 88, torch.bfloat16
    gen = _gen(15)
    X, Y = _ints(gen, (131, P), dt), _ints(gen, (131, Q), dt)
    want = _ref_wgrad(X, Y, edges)
    if pad_x:
        X = _padded(X, P + pad_x)
    if pad_y:
        Y = _padded(Y, Q + pad_y)
    if off:
        flat = torch.full((131 * Q + off,), float("nan"), dtype=dt, device="cuda")
        flat[off:] = Y.reshape(-1)
        Y = flat[off:].view(131, Q)
    full = torch.full((3, P + 1, Q + 3), 5.0, device="cuda")
    out = full[:, :P, :Q]
    _ops().gemm_grouped_wgrad(X, Y, _dev(edges), "f32", out=out)
    assert torch.equal(out.double(), want)
    _ops().gemm_grouped_wgrad(X, Y, _dev(edges), "f32", out=out, alpha=0.5, beta=1.0)  # adds to what is held
    assert torch.equal(out.double(), 1.5 * want)
    _ops().gemm_grouped_wgrad(X, Y, _dev(edges), "f32", out=out, alpha=0.0, beta=2.0)
    assert torch.equal(out.double(), 3.0 * want)
    assert (full[:, P:] == 5).all() and (full[:, :, Q:] == 5).all()
    half = torch.full((3, P, Q), float("nan"), dtype=dt, device="cuda")
    _ops().gemm_grouped_wgrad(X[:0], Y[:0], _dev([0, 0, 0, 0]), "bf16", out=half)
    assert (half == 0).all()


# ---- both together ---------------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_gradients_of_an_expert_layer(layout):
    """One layer's forward product and both gradients, as a training step uses them: against the
    formula in 64 bits, and the loss sum(C·G) against differences (it is linear in each operand, so
    with small integers the difference of two evaluations is the derivative exactly)."""
    edges, N, K, dt = _offsets([37, 0, 64, 5], 0), 56, 40, torch.bfloat16
    M, gen, ops = edges[-1], _gen(21), _ops()
    off = _dev(edges)
    A, G = _ints(gen, (M, K), dt), _ints(gen, (M, N), dt)
    B = _ints(gen, (4, K, N) if layout == "kn" else (4, N, K), dt)
    other = "nk" if layout == "kn" else "kn"
    C = ops.gemm_grouped(A, B, off, layout, "f32")
    dA = ops.gemm_grouped(G, B, off, other, "f32")
    dB = ops.gemm_grouped_wgrad(A, G, off) if layout == "kn" else ops.gemm_grouped_wgrad(G, A, off)
    a, b = A.double().requires_grad_(), B.double().requires_grad_()
    rows = [a[lo:hi] @ (b[e] if layout == "kn" else b[e].t()) for e, (lo, hi) in enumerate(zip(edges, edges[1:]))]
    loss = (torch.cat(rows) * G.double()).sum()
    loss.backward()
    assert torch.equal(C.double(), torch.cat(rows).detach())
    assert torch.equal(dA.double(), a.grad) and torch.equal(dB.double(), b.grad)

    def value(x, y):
        return (ops.gemm_grouped(x, y, off, layout, "f32").double() * G.double()).sum().item()

    base = value(A, B)
    for r, c in ((0, 0), (36, 39), (37, 5), (M - 1, 17)):
        x = A.clone()
        x[r, c] += 1
        assert value(x, B) - base == dA[r, c].item()
    for e, r, c in ((0, 0, 0), (1, 3, 3), (2, 39, 39), (3, 7, 11)):
        y = B.clone()
        y[e, r, c] += 1
        assert value(A, y) - base == dB[e, r, c].item()


@gpu
def test_replayed_graph_reads_the_offsets_it_finds():
    """Forward and gradients captured once and replayed with other offsets and other rows, eager work
    in between; every replay equals the eager result."""
    ops, dt, gen = _ops(), torch.bfloat16, _gen(31)
    M, N, K, G = 300, 72, 104, 5
    A, D = _ints(gen, (M, K), dt), _ints(gen, (M, N), dt)
    B, off = _ints(gen, (G, N, K), dt), _dev([0, 10, 60, 60, 200, 300])
    C, dA, dB = (torch.zeros(s, device="cuda") for s in ((M, N), (M, K), (G, N, K)))

    def work(c, da, db):
        ops.gemm_grouped(A, B, off, "nk", "f32", out=c)
        ops.gemm_grouped(D, B, off, "kn", "f32", out=da)
        ops.gemm_grouped_wgrad(D, A, off, "f32", out=db)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(C, dA, dB)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(C, dA, dB)
    for edges in ([0, 10, 60, 60, 200, 300], [0, 0, 0, 300, 300, 300], [5, 80, 81, 150, 150, 299], [0, 1, 2, 3, 4, 5]):
        off.copy_(_dev(edges))
        A.copy_(_ints(gen, (M, K), dt))
        for t in (C, dA, dB):
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        c, da, db = (torch.full_like(t, 9.0) for t in (C, dA, dB))
        work(c, da, db)
        assert torch.equal(C, c) and torch.equal(dA, da) and torch.equal(dB, db)
        lo, hi = edges[0], edges[-1]
        assert torch.equal(C[lo:hi].double(), _ref_rows(A, B, edges, "nk")[lo:hi])
        assert torch.equal(dB.double(), _ref_wgrad(D, A, edges))


@gpu
def test_two_streams_at_once():
    """Calls that repack, on two streams and the current one, each with the workspace it allocates."""
    ops, dt, gen = _ops(), torch.bfloat16, _gen(41)
    edges, N, K = _offsets([100, 200, 84], 0), 131, 99
    A = [_ints(gen, (384, K), dt) for _ in range(2)]
    B, off = _ints(gen, (3, K, N), dt), _dev(edges)
    want = [_ref_rows(a, B, edges, "kn").float() for a in A]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for i in range(6):
        got.append(ops.gemm_grouped(A[i % 2], B, off, "kn", "f32", stream=streams[i % 2]))
        got.append(ops.gemm_grouped(A[i % 2], B, off, "kn", "f32"))
    torch.cuda.synchronize()
    for i in range(6):
        assert torch.equal(got[2 * i], want[i % 2]) and torch.equal(got[2 * i + 1], want[i % 2])


@gpu
def test_offsets_out_of_order_or_range_stay_inside_the_operands():
    ops, dt, gen = _ops(), torch.bfloat16, _gen(51)
    A, B = _ints(gen, (64, 48), dt), _ints(gen, (3, 48, 40), dt)
    out = torch.full((66, 40), 7.0, device="cuda")
    for edges, good in (([-5, 10, 20, 1 << 30], [0, 10, 20, 64]), ([0, 30, 12, 12], [0, 30, 30, 30]),
                        ([70, 80, 90, 100], [64, 64, 64, 64])):
        out.fill_(7.0)
        ops.gemm_grouped(A, B, _dev(edges), "kn", "f32", out=out[1:65])
        want = _ref_rows(A, B, good, "kn")
        assert torch.equal(out[1 + good[0]:1 + good[-1]].double(), want[good[0]:good[-1]])
        assert (out[0] == 7).all() and (out[65] == 7).all() and (out[1 + good[-1]:] == 7).all()
        g = ops.gemm_grouped_wgrad(A, A, _dev(edges))
        assert torch.equal(g.double(), _ref_wgrad(A, A, good))


@gpu
@pytest.mark.parametrize("groups,rows,empty_every", [(1000, 3000, 3), (4096, 5000, 2), (65, 64, 0)])
def test_many_groups(groups, rows, empty_every):
    gen, dt = _gen(groups), torch.bfloat16
    rng = np.random.default_rng(groups)
    sizes = rng.multinomial(rows, np.ones(groups) / groups)
    if empty_every:
        sizes[::empty_every] = 0
    edges = _offsets(sizes, 2)
    A, B = _ints(gen, (edges[-1] + 3, 24), dt), _ints(gen, (groups, 16, 24), dt)
    want = _ref_rows(A, B, edges, "nk")
    out = _ops().gemm_grouped(A, B, _dev(edges), "nk", "f32", out=torch.zeros((edges[-1] + 3, 16), device="cuda"))
    assert torch.equal(out.double(), want)
    g = _ops().gemm_grouped_wgrad(A, A, _dev(edges))
    assert torch.equal(g.double(), _ref_wgrad(A, A, edges))


@gpu
def test_offsets_past_32_bits():
    """Rows at the largest pitch and matrices 4 GiB apart: operands whose byte offsets pass 2^32, laid
    over one buffer with NaN where nothing may be read (small enough pieces are written)."""
    dt, gen = torch.bfloat16, _gen(61)
    pitch, M, N, K = (1 << 22) - 8, 600, 24, 40  # 600 rows of 8 MiB: 5 GB
    buf = torch.empty(pitch * M, dtype=dt, device="cuda")
    A = buf.as_strided((M, K), (pitch, 1))
    A.copy_(_ints(gen, (M, K), dt))
    B = _ints(gen, (2, N, K), dt)
    edges = [0, 590, 600]
    out = _ops().gemm_grouped(A, B, _dev(edges), "nk", "f32")
    assert torch.equal(out.double(), _ref_rows(A, B, edges, "nk"))
    g = _ops().gemm_grouped_wgrad(A, _ints(gen, (M, N), dt), _dev(edges))
    assert g.isfinite().all()
    Y = _ints(gen, (M, N), dt)
    assert torch.equal(_ops().gemm_grouped_wgrad(Y, A, _dev(edges)).double(), _ref_wgrad(Y, A, edges))
    for layout, shape in (("nk", (N, K)), ("kn", (K, N))):
        stride = (1 << 31) + 64  # elements: the second matrix lies 4 GiB and a little behind
        W = buf.as_strided((2, *shape), (stride, shape[1], 1))
        W.copy_(_ints(gen, (2, *shape), dt))
        X = _ints(gen, (30, K), dt)
        out = _ops().gemm_grouped(X, W, _dev([0, 11, 30]), layout, "f32")
        assert torch.equal(out.double(), _ref_rows(X, W, [0, 11, 30], layout))
    C = buf.view(torch.float32).as_strided((2, N, K), ((1 << 30) + 128, K, 1))
    X, Y = _ints(gen, (30, N), dt), _ints(gen, (30, K), dt)
    _ops().gemm_grouped_wgrad(X, Y, _dev([0, 11, 30]), "f32", out=C)
    assert torch.equal(C.double(), _ref_wgrad(X, Y, [0, 11, 30]))


@gpu
def test_torch_helper_refusals():
    ops, dt = _ops(), torch.bfloat16
    A, B = torch.zeros((8, 16), dtype=dt, device="cuda"), torch.zeros((2, 16, 24), dtype=dt, device="cuda")
    off = _dev([0, 3, 8])
    bad = [
        (A.float(), B, off, {}), (A, B.half(), off, {}), (A[:, :8], B, off, {}), (A, B[:1], off, {}),
        (A, B, off.long(), {}), (A, B, off.cpu(), {}), (A.cpu(), B, off, {}), (A, B[0], off, {}),
        (A, B, off, dict(b_layout="nn")), (A, B, off, dict(out_dtype="f16")),
        (A, B, off, dict(out=torch.zeros((8, 25), device="cuda"), out_dtype="f32")),
        (A, B, off, dict(out=torch.zeros((8, 24), device="cuda"))),
        (A, B.transpose(1, 2), off, dict(b_layout="nk")),
    ]
    for a, b, o, kw in bad:
        with pytest.raises(ValueError):
            ops.gemm_grouped(a, b, o, **kw)
    with pytest.raises(tbg.Error):
        ops.gemm_grouped(A, B[:1].expand(2, 16, 24), off)
    for x, y, o, kw in ((A, A[:4], off, {}), (A, A.half(), off, {}), (A, A, off, dict(out_dtype="f16")),
                        (A, A, off, dict(out=torch.zeros((2, 16, 15), device="cuda")))):
        with pytest.raises(ValueError):
            ops.gemm_grouped_wgrad(x, y, o, **kw)


# Offsets that descend: the pairs together claim more tiles than groups that ascend can make.
DESCENDING = [
    (1000, [0, 900, 0, 900, 0, 900, 1000]),
    (2000, [0, 1900, 0, 2000]),
    (40, [0, 36, 0, 36, 0, 40]),
    (3000, [0, 2990] * 100 + [0, 3000]),
    (700, [100, 600, -7, 90] + [650, 20] * 40 + [1 << 30, 600, 640, 5]),
]


@gpu
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("M,edges", DESCENDING)
def test_rows_of_descending_offsets_belong_to_the_first_group_that_reaches_them(M, edges, layout):
    """An offset below an earlier one counts as that one, so every row up to the largest offset has one
    group, and none is left out."""
    print(f"rows {layout} descending offsets M={M} groups={len(edges) - 1}", flush=True)
    gen, dt, G, K = _gen(M), torch.bfloat16, len(edges) - 1, 72
    good = np.maximum.accumulate(np.clip(edges, 0, M)).tolist()
    for N in (40, 1032):
        A, B = _ints(gen, (M, K), dt), _ints(gen, (G, K, N) if layout == "kn" else (G, N, K), dt)
        out = torch.full((M + 2, N), 7.0, device="cuda")
        _ops().gemm_grouped(A, B, _dev(edges), layout, "f32", out=out[1:M + 1])
        want = torch.full((M + 2, N), 7.0, device="cuda")
        want[1 + good[0]:1 + good[-1]] = _ref_rows(A, B, good, layout)[good[0]:good[-1]].float()
        assert torch.equal(out, want), N


@gpu
@pytest.mark.parametrize("layout", ["nk", "kn"])
def test_one_row_at_any_pitch(layout):
    """The last token of one sequence: a single row whose stride in the hidden states, never used, passes
    the largest leading dimension; matrices of a single row likewise, and the weight gradient."""
    gen, dt, K, N = _gen(77), torch.bfloat16, 4096, 40
    hidden = _ints(gen, (1, 1100, K), dt)
    A = hidden[:, -1]
    assert A.stride(0) >= 1 << 22
    B = _ints(gen, (1, N, K) if layout == "nk" else (1, K, N), dt)
    out = _ops().gemm_grouped(A, B, _dev([0, 1]), layout, "f32")
    assert torch.equal(out.double(), _ref_rows(A, B, [0, 1], layout))
    grad = _ops().gemm_grouped_wgrad(A, out.to(dt), _dev([0, 1]))
    assert torch.equal(grad.double(), _ref_wgrad(A, out.to(dt), [0, 1]))
    wide = torch.full((2, 1, 1 << 23), float("nan"), dtype=dt, device="cuda")
    X = _ints(gen, (9, 24), dt)
    one = wide[:, :, :24] if layout == "nk" else wide[:, :, :16]
    one.copy_(_ints(gen, one.shape, dt))
    X = X if layout == "nk" else X[:, :1]
    got = _ops().gemm_grouped(X, one, _dev([0, 4, 9]), layout, "f32")
    assert torch.equal(got.double(), _ref_rows(X, one, [0, 4, 9], layout))
    C = torch.full((1, 1, 1 << 23), 5.0, device="cuda")[:, 0, :N]
    _ops().gemm_grouped(A, B, _dev([0, 1]), layout, "f32", out=C)
    assert torch.equal(C, out)


@gpu
def test_a_sum_with_c_needs_c():
    """beta·C without the matrix that holds C would add what new memory happens to hold."""
    ops, dt = _ops(), torch.bfloat16
    A, B, off = torch.ones((8, 32), dtype=dt, device="cuda"), torch.ones((2, 24, 32), dtype=dt, device="cuda"), _dev([0, 3, 8])
    (a, sa), (b, sb) = ops.mx4_quantize(A), ops.mx4_quantize(B)
    for call in (lambda **k: ops.gemm_grouped(A, B, off, "nk", **k), lambda **k: ops.gemm_grouped_wgrad(A, A, off, **k),
                 lambda **k: ops.mx4_gemm(a, sa, b[0], sb[0], **k), lambda **k: ops.mx4_gemm_grouped(a, sa, b, sb, off, **k)):
        with pytest.raises(ValueError, match="beta"):
            call(beta=1.0)
        assert call(beta=0.0).isfinite().all()


@gpu
def test_a_refused_call_enqueues_nothing():
    """2^24 workgroups of 64 columns over rows that need a repack (K = 1): refused as unsupported, and the
    workspace is as it was."""
    N = 1 << 30
    A, B = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda"), torch.ones((1, N, 1), dtype=torch.bfloat16, device="cuda")
    C = torch.empty((1, N), dtype=torch.bfloat16, device="cuda")
    need = tbg.gemm_grouped_workspace_query(1, 1, N, 1, "bf16", A.data_ptr(), 1, B.data_ptr(), 1, N, "nk")
    assert need > 16 * N
    ws = torch.full((need // 8,), 0x5A5A5A5A, dtype=torch.int64, device="cuda")
    with pytest.raises(tbg.Error) as e:
        _ops().gemm_grouped(A, B, _dev([0, 1]), "nk", "bf16", out=C, workspace=ws)
    assert e.value.status == tbg.ERR_UNSUPPORTED, e.value
    torch.cuda.synchronize()
    assert all((part == 0x5A5A5A5A).all() for part in ws.split(1 << 26))


@gpu
def test_repacks_of_more_than_64_gib_together():
    """Rows of 1025 values, 16.7 million of them: both operands of the weight gradient are repacked, 32 GiB
    each, more than the chunks that one launch numbers.  The groups are a few rows at the far end."""
    M, P, dt, gen = (1 << 24) + 5, 1025, torch.bfloat16, _gen(91)
    edges = [M - 200, M - 150, M - 150, M - 3]
    X, Y = (torch.empty((M, P), dtype=dt, device="cuda") for _ in range(2))
    for t in (X, Y):
        t[M - 300:] = _ints(gen, (300, P), dt)
    need = tbg.gemm_grouped_wgrad_workspace_query(3, M, P, P, "bf16", X.data_ptr(), P, Y.data_ptr(), P)
    assert need > 64 << 30
    out = _ops().gemm_grouped_wgrad(X, Y, _dev(edges), workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    far = slice(M - 300, M)
    assert torch.equal(out.double(), _ref_wgrad(X[far], Y[far], [e - (M - 300) for e in edges]))
    del X, Y
    torch.cuda.empty_cache()


@gpu
@pytest.mark.parametrize("groups,dtype", [(64, "bf16"), (64, "f16"), (5, "bf16"), (2, "f16")])
def test_wgrad_exact_in_the_order_of_the_rows(groups, dtype):
    """1024 rows a group on average, up to 64 groups: the groups run longest first.  Equal ones, empty ones
    and one of most of the rows."""
    sizes = ([900, 0, 1100, 900] * groups)[:groups]
    sizes[groups // 2] += 1024 * groups - sum(sizes) + 8
    edges, P, Q, dt = _offsets(sizes, 3), 137, 72, TORCH[dtype]
    M, gen = edges[-1] + 5, _gen(groups)
    X, Y = _ints(gen, (M, P), dt), _ints(gen, (M, Q), dt)
    want = _ref_wgrad(X, Y, edges)
    for t in (X, Y):
        t[:3], t[edges[-1]:] = float("nan"), float("nan")
    out = torch.full((groups, P, Q), float("nan"), device="cuda")
    _ops().gemm_grouped_wgrad(X, Y, _dev(edges), out=out)
    assert torch.equal(out.double(), want)
