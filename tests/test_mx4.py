"""Microscaled 4-bit data: quantisation, the way back, and the products, dense and over ragged groups.

Quantisation and decoding are exact definitions: codes, scale bytes and values must equal the
reference (written from the format's fields, in 64 bits) bit for bit.  The products' operands have
codes of all sixteen kinds and scales 2^-1..2^1, so every term is a multiple of 1/16 below 144 and a
sum of K <= 1024 of them is below 2^24 sixteenths: fp32 holds it exactly whatever the order, and the
output must equal the reference rounded once.  Products of operands with a wide spread of scales are
held to the bound of an fp32 sum: K·2^-23·sum|a·b| + eps/2·(|exact| + that)."""
import numpy as np
import pytest
import torch

import tiled_bf16_gemm_amd as tbg

gpu = pytest.mark.gpu
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
PTR = 0x7F00_0000_0000


def _ops():
    from tiled_bf16_gemm_amd import torch_ops
    return torch_ops


# ---- the reference (numpy, 64 bits) ----------------------------------------------------------------

def ref_quantize(x):
    """Codes (rows, K) and scale bytes (rows, K/32) of x (rows, cols), K = cols rounded up to 32."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    v = np.zeros((rows, -(-cols // 32) * 32))
    v[:, :cols] = x
    v = v.reshape(rows, -1, 32)
    bad = ~np.isfinite(v).all(-1)
    m = np.where(bad, 0.0, np.abs(v).max(-1, initial=0.0))
    e = np.where(m > 0, np.frexp(np.where(m > 0, m, 1.0))[1] - 1, -1000) - 2
    e = np.clip(e, -127, 127)
    a = np.abs(np.where(bad[..., None], 0.0, v)) / np.exp2(e.astype(np.float64))[..., None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    code = np.zeros(a.shape, dtype=np.uint8)
    for i, b in enumerate(mid):  # a tie goes to the even code: up at mid points 1, 3, 5
        code += ((a >= b) if i % 2 else (a > b)).astype(np.uint8)
    code |= (np.signbit(v) & ~bad[..., None]).astype(np.uint8) << 3
    return code.reshape(rows, -1), np.where(bad, 255, e + 127).astype(np.uint8)


def ref_values(code, scale):
    c = np.asarray(code, dtype=np.int64)
    mag = GRID[c & 7] * np.where(c & 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, np.exp2(scale.astype(np.float64) - 127))
    return mag * np.repeat(s, 32, axis=-1)


def pack(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def unpack(codes):
    out = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = codes & 15, codes >> 4
    return out


def test_reference_on_hand_worked_blocks():
    """The reference itself: a block with maximum 6 (scale 1), its ties, and a block scaled by 1/4."""
    x = np.zeros((1, 64))
    x[0, :14] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.26, -0.0, 4.9, 5.1]
    x[0, 32:36] = [1.9, -1.0, 0.0625, 0.125]
    code, scale = ref_quantize(x)
    assert scale.tolist() == [[127, 125]]
    assert code[0, :14].tolist() == [7, 15, 0, 2, 2, 4, 4, 6, 6, 14, 1, 8, 6, 7]
    assert code[0, 32:36].tolist() == [7, 14, 0, 1]  # 7.6 clips to 6, -4, 0.25 ties to 0, 0.5
    v = ref_values(code, scale)
    assert v[0, 0] == 6 and v[0, 32] == 1.5 and v[0, 33] == -1.0 and v[0, 35] == 0.125
    assert (unpack(pack(code)) == code).all()


# ---- refusals (CPU) --------------------------------------------------------------------------------

def _q(**over):
    a = dict(rows=4, cols=40, X=PTR, ldx=40, x_dtype="bf16", codes=PTR, ld_codes=32, scales=PTR, ld_scales=16)
    a.update(over)
    return a


@pytest.mark.parametrize("fn", ["mx4_quantize", "mx4_dequantize"])
@pytest.mark.parametrize("over,status", [
    (dict(rows=-1), tbg.ERR_INVALID_VALUE),
    (dict(cols=-1), tbg.ERR_INVALID_VALUE),
    (dict(x_dtype="u8"), tbg.ERR_INVALID_VALUE),
    (dict(ldx=39), tbg.ERR_INVALID_VALUE),
    (dict(X=0), tbg.ERR_INVALID_VALUE),
    (dict(X=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(X=PTR + 2, x_dtype="f32"), tbg.ERR_MISALIGNED),
    (dict(codes=0), tbg.ERR_INVALID_VALUE),
    (dict(scales=0), tbg.ERR_INVALID_VALUE),
    (dict(ld_codes=16), tbg.ERR_INVALID_VALUE),
    (dict(ld_scales=0), tbg.ERR_INVALID_VALUE),
    (dict(ld_codes=40), tbg.ERR_MISALIGNED),
    (dict(ld_scales=8), tbg.ERR_MISALIGNED),
    (dict(codes=PTR + 8), tbg.ERR_MISALIGNED),
    (dict(scales=PTR + 4), tbg.ERR_MISALIGNED),
    (dict(cols=(1 << 30) + 1, ldx=1 << 31, ld_codes=1 << 30, ld_scales=1 << 26), tbg.ERR_UNSUPPORTED),
])
def test_conversion_refusals(fn, over, status):
    with pytest.raises(tbg.Error) as e:
        getattr(tbg, fn)(**_q(**over))
    assert e.value.status == status, e.value


def _p(**over):
    a = dict(M=4, N=8, K=64, alpha=1.0, A=PTR, lda=32, A_scales=PTR, ld_as=16, B=PTR, ldb=32, B_scales=PTR, ld_bs=16,
             beta=0.0, C=PTR, ldc=8, c_dtype="f32")
    a.update(over)
    return a


BAD_PRODUCT = [
    (dict(M=-1), tbg.ERR_INVALID_VALUE),
    (dict(K=65), tbg.ERR_INVALID_VALUE),
    (dict(K=48), tbg.ERR_INVALID_VALUE),
    (dict(N=(1 << 30) + 1, ldc=1 << 31), tbg.ERR_UNSUPPORTED),
    (dict(lda=16), tbg.ERR_INVALID_VALUE),
    (dict(ldb=16), tbg.ERR_INVALID_VALUE),
    (dict(ld_as=0), tbg.ERR_INVALID_VALUE),
    (dict(lda=40), tbg.ERR_MISALIGNED),
    (dict(ld_bs=8), tbg.ERR_MISALIGNED),
    (dict(A=PTR + 8), tbg.ERR_MISALIGNED),
    (dict(B_scales=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(lda=1 << 23), tbg.ERR_UNSUPPORTED),
    (dict(ldc=7), tbg.ERR_INVALID_VALUE),
    (dict(c_dtype="f16"), tbg.ERR_INVALID_VALUE),
    (dict(A=0), tbg.ERR_INVALID_VALUE),
    (dict(B_scales=0), tbg.ERR_INVALID_VALUE),
    (dict(C=0), tbg.ERR_INVALID_VALUE),
]


@pytest.mark.parametrize("over,status", BAD_PRODUCT)
def test_product_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.mx4_gemm(**_p(**over))
    assert e.value.status == status, e.value


@pytest.mark.parametrize("over,status", BAD_PRODUCT + [
    (dict(groups=-1), tbg.ERR_INVALID_VALUE),
    (dict(groups=4097), tbg.ERR_UNSUPPORTED),
    (dict(offsets=0), tbg.ERR_INVALID_VALUE),
    (dict(offsets=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(stride_b=8 * 32 - 16), tbg.ERR_INVALID_VALUE),
    (dict(stride_bs=0), tbg.ERR_INVALID_VALUE),
    (dict(stride_b=8 * 32 + 8), tbg.ERR_MISALIGNED),
])
def test_grouped_product_refusals(over, status):
    a = dict(_p(), groups=2, offsets=PTR, stride_b=8 * 32, stride_bs=8 * 16)
    a.update(over)
    with pytest.raises(tbg.Error) as e:
        tbg.mx4_gemm_grouped(**a)
    assert e.value.status == status, e.value


@pytest.mark.gpu
def test_more_tiles_than_a_launch_takes_are_refused():
    """2^24 workgroups of 64 columns: refused on the host, nothing is launched."""
    with pytest.raises(tbg.Error) as e:
        tbg.mx4_gemm(**_p(M=1, N=1 << 30, K=32, lda=16, ldb=16, ldc=1 << 30))
    assert e.value.status == tbg.ERR_UNSUPPORTED, e.value


def test_empty_calls_need_no_device():
    tbg.mx4_quantize(**_q(rows=0, X=0, codes=0, scales=0))
    tbg.mx4_dequantize(**_q(cols=0, X=0, codes=0, scales=0))
    tbg.mx4_gemm(**_p(M=0, A=0, A_scales=0, C=0))
    tbg.mx4_gemm_grouped(**dict(_p(), groups=0, offsets=0, stride_b=0, stride_bs=0))


# ---- quantisation ----------------------------------------------------------------------------------

def _quantize(x, **kw):
    codes, scales = _ops().mx4_quantize(x, **kw)
    return unpack(codes.cpu().numpy()), scales.cpu().numpy()


def _check_quantize(x):
    code, scale = _quantize(x)
    want_code, want_scale = ref_quantize(x.double().cpu().numpy())
    assert (scale == want_scale).all()
    assert (code == want_code).all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (7, 2049), (5, 31), (64, 256), (130, 1000), (2, 8191)])
def test_quantize_and_back(rows, cols, dtype):
    gen = torch.Generator(device="cuda").manual_seed(rows * 10007 + cols)
    spread = torch.exp(2 * torch.randn((rows, 1), generator=gen, device="cuda"))
    x = (torch.randn((rows, cols), generator=gen, device="cuda") * spread).to(TORCH[dtype])
    _check_quantize(x)
    codes, scales = _ops().mx4_quantize(x)
    want = ref_values(*ref_quantize(x.double().cpu().numpy()))[:, :cols]
    for out_dtype in ("f32", "bf16", "f16"):
        if out_dtype == "f16" and np.abs(want).max() > 60000:
            continue
        v = _ops().mx4_dequantize(codes, scales, cols=cols, out_dtype=out_dtype)
        assert torch.equal(v.cpu(), torch.from_numpy(want).to(TORCH[out_dtype]))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize_ties_borders_and_extremes(dtype):
    """Every tie and its neighbours at many scales, the type's largest, smallest and subnormal values,
    zeros, and blocks with a NaN or an infinity."""
    dt, info = TORCH[dtype], torch.finfo(TORCH[dtype])
    rows = []
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    step = {"bf16": 2.0 ** -7, "f16": 2.0 ** -10, "f32": 2.0 ** -23}[dtype]
    for e in (-14, -6, 0, 3, 9):
        base = [4.0] + [s * m * f for m in mids for s in (1, -1) for f in (1, 1 + step)] + [7.0, -7.5, 0.0]
        rows.append([v * 2.0 ** e for v in base])
    rows.append([info.max, -info.max, info.max / 2, 1.0] + [0.0] * 28)
    rows.append([info.tiny, -info.tiny / 2, info.tiny / 4] + [0.0] * 29)
    rows.append([info.smallest_normal * info.eps] * 3 + [0.0] * 29)
    rows.append([0.0] * 31 + [-0.0])
    for v in (float("nan"), float("inf"), float("-inf")):
        rows.append([1.0, 2.0, v] + [3.0] * 29)
    x = torch.tensor([r[:32] + [0.0] * (32 - len(r)) for r in rows], dtype=torch.float64).to(dt).cuda()
    _check_quantize(x)
    codes, scales = _ops().mx4_quantize(x)
    v = _ops().mx4_dequantize(codes, scales, out_dtype="f32").cpu()
    assert v[-3:].isnan().all() and v[:-3].isfinite().all()
    for out_dtype in ("bf16", "f16"):
        assert _ops().mx4_dequantize(codes, scales, out_dtype=out_dtype).cpu()[-3:].isnan().all()


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_strides_stacks_and_padding(dtype):
    dt = TORCH[dtype]
    gen = torch.Generator(device="cuda").manual_seed(3)
    full = torch.full((3, 50, 75), float("nan"), device="cuda").to(dt)
    full[:, :, 1:71] = torch.randn((3, 50, 70), generator=gen, device="cuda").to(dt)
    x = full[:, :, 1:71]
    want_code, want_scale = ref_quantize(x.double().cpu().numpy().reshape(150, 70))
    # into the caller's buffers: what lies between the rows stays
    codes = torch.full((3, 50, 64), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((3, 50, 16), 0xCD, dtype=torch.uint8, device="cuda")
    _ops().mx4_quantize(x, codes[..., :48], scales[..., :3])
    assert (unpack(codes[..., :48].cpu().numpy()).reshape(150, -1) == want_code).all()
    assert (scales[..., :3].cpu().numpy().reshape(150, -1) == want_scale).all()
    assert (codes[..., 48:] == 0xAB).all() and (scales[..., 3:] == 0xCD).all()
    out = torch.full((3, 50, 75), 7.0, device="cuda")
    _ops().mx4_dequantize(codes[..., :48], scales[..., :3], cols=70, out_dtype="f32", out=out[..., 2:72])
    want = ref_values(want_code, want_scale)[:, :70].reshape(3, 50, 70)
    assert (out[..., 2:72].cpu().numpy() == want).all()
    assert (out[..., :2] == 7).all() and (out[..., 72:] == 7).all()
    one_code, one_scale = _quantize(x[:, :1])
    assert (one_code.reshape(3, -1) == want_code[::50]).all() and (one_scale.reshape(3, -1) == want_scale[::50]).all()


# ---- products --------------------------------------------------------------------------------------

def _random_mx4(rng, shape, K, spread=1, pitch_codes=0, pitch_scales=16):
    """Random codes and scales with rows at a pitch, the padding set to what must not be used (codes
    of 6, NaN scales): the torch views, and the values in 64 bits."""
    code = rng.integers(0, 16, (*shape, K)).astype(np.uint8)
    scale = rng.integers(127 - spread, 128 + spread, (*shape, K // 32)).astype(np.uint8)
    ld_c, ld_s = K // 2 + pitch_codes, -(-(K // 32) // 16) * 16 + pitch_scales
    held_c = np.full((*shape, ld_c), 0x77, dtype=np.uint8)
    held_s = np.full((*shape, ld_s), 255, dtype=np.uint8)
    held_c[..., :K // 2], held_s[..., :K // 32] = pack(code), scale
    c = torch.from_numpy(held_c).cuda()[..., :K // 2]
    s = torch.from_numpy(held_s).cuda()[..., :K // 32]
    return c, s, torch.from_numpy(ref_values(code, scale)).cuda()


# one row; one block; K ends inside a tile of 256, of 512; sizes that overhang and take each tile
PRODUCTS = [(1, 1, 32), (1, 16, 64), (1, 300, 1024), (3, 40, 288), (16, 130, 224), (17, 70, 256), (64, 64, 512),
            (33, 129, 544), (65, 200, 736), (200, 520, 320), (300, 1030, 800), (1030, 2050, 96), (2100, 2056, 288),
            (4100, 4100, 160), (20, 70001, 96), (50, 70001, 288)]


@gpu
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product_exact(M, N, K):
    print(f"mx4 product M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(M * 31 + N * 7 + K)
    a, sa, va = _random_mx4(rng, (M,), K, pitch_codes=16)
    b, sb, vb = _random_mx4(rng, (N,), K)
    want = va @ vb.t().contiguous()
    for out_dtype in ("f32", "bf16"):
        full = torch.full((M + 1, N + 3), -9.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().mx4_gemm(a, sa, b, sb, out_dtype, out=full[:M, :N])
        assert torch.equal(full[:M, :N], want.to(full.dtype)), out_dtype
        assert (full[M] == -9).all() and (full[:, N:] == -9).all()


@gpu
@pytest.mark.parametrize("M,N,K", [(1, 500, 4096), (20, 300, 2080), (300, 400, 3104), (1100, 900, 1184)])
def test_product_of_wide_scales(M, N, K):
    rng = np.random.default_rng(K)
    a, sa, va = _random_mx4(rng, (M,), K, spread=12)
    b, sb, vb = _random_mx4(rng, (N,), K, spread=12)
    want, mag = va @ vb.t().contiguous(), va.abs() @ vb.abs().t().contiguous()
    for out_dtype in ("f32", "bf16"):
        out = _ops().mx4_gemm(a, sa, b, sb, out_dtype)
        acc = K * 2.0 ** -23 * mag
        bound = acc + torch.finfo(out.dtype).eps / 2 * (want.abs() + acc)
        assert ((out.double() - want).abs() <= bound).all()


@gpu
@pytest.mark.parametrize("M,N", [(1, 48), (70, 48), (300, 700), (1300, 1500)])
def test_product_alpha_beta_and_empty_sum(M, N):
    rng, K = np.random.default_rng(7), 352
    a, sa, va = _random_mx4(rng, (M,), K)
    b, sb, vb = _random_mx4(rng, (N,), K)
    S = va @ vb.t().contiguous()
    C = torch.from_numpy(rng.integers(-8, 9, (M, N)).astype(np.float32)).cuda()
    for out_dtype in ("f32", "bf16"):
        for alpha, beta in ((0.5, 0.0), (1.0, 1.0), (-2.0, 0.25), (0.0, 2.0), (0.0, 0.0)):
            out = C.to(TORCH[out_dtype], copy=True) if beta else torch.full((M, N), float("nan"), dtype=TORCH[out_dtype], device="cuda")
            _ops().mx4_gemm(a, sa, b, sb, out_dtype, out=out, alpha=alpha, beta=beta)
            want = alpha * S + (beta * C.double() if beta else 0.0)
            assert torch.equal(out, want.to(out.dtype)), (out_dtype, alpha, beta)
        none = torch.full((M, N), float("nan"), dtype=TORCH[out_dtype], device="cuda")
        _ops().mx4_gemm(a[:, :0], sa[:, :0], b[:, :0], sb[:, :0], out_dtype, out=none)
        assert (none == 0).all()


@gpu
@pytest.mark.parametrize("M", [2, 100, 400])
def test_nan_blocks_reach_their_rows_and_columns_only(M):
    rng, N, K = np.random.default_rng(17), 90, 320
    a, sa, va = _random_mx4(rng, (M,), K)
    b, sb, vb = _random_mx4(rng, (N,), K)
    want = (va @ vb.t().contiguous()).float()
    sa[1, 9], sb[4, 0] = 255, 255
    out = _ops().mx4_gemm(a, sa, b, sb, "f32")
    rows, cols = torch.ones(M, dtype=torch.bool), torch.ones(N, dtype=torch.bool)
    rows[1], cols[4] = False, False
    assert torch.equal(out[rows][:, cols], want[rows][:, cols])
    assert out[1].isnan().all() and out[:, 4].isnan().all()


GROUPED = [
    ([1], 0, 0, 16, 32),
    ([0, 0], 0, 3, 40, 64),
    ([3, 0, 1, 0, 7], 1, 4, 40, 288),
    ([1] * 70 + [0] * 3 + [9], 0, 1, 130, 544),
    ([5, 64, 0, 65, 1], 2, 3, 131, 96),
    ([130, 0, 257, 700], 0, 9, 520, 192),
    ([900, 1200, 0, 133], 1, 0, 1030, 736),
    ([2100, 1900], 0, 17, 4100, 160),
]


@gpu
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_product_exact(case):
    sizes, before, behind, N, K = GROUPED[case]
    edges = [before] + [before + int(v) for v in np.cumsum(sizes)]
    M, G = edges[-1] + behind, len(sizes)
    print(f"mx4 grouped product groups={G} M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(case)
    a, sa, va = _random_mx4(rng, (M,), K)
    b, sb, vb = _random_mx4(rng, (G, N), K, pitch_codes=16)
    want = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for e in range(G):
        want[edges[e]:edges[e + 1]] = va[edges[e]:edges[e + 1]] @ vb[e].t().contiguous()
    for e, n in enumerate(sizes):
        if n == 0:
            sb[e] = 255
    sa[:before], sa[edges[-1]:] = 255, 255
    off = torch.tensor(edges, dtype=torch.int32, device="cuda")
    for out_dtype in ("f32", "bf16"):
        out = torch.full((M, N), -9.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().mx4_gemm_grouped(a, sa, b, sb, off, out_dtype, out=out)
        assert torch.equal(out[before:edges[-1]], want[before:edges[-1]].to(out.dtype)), out_dtype
        assert (out[:before] == -9).all() and (out[edges[-1]:] == -9).all()
    out = torch.full((M, N), 3.0, device="cuda")
    _ops().mx4_gemm_grouped(a, sa, b, sb, off, "f32", out=out, alpha=0.5, beta=2.0)
    assert torch.equal(out[before:edges[-1]].double(), 0.5 * want[before:edges[-1]] + 6)


@gpu
@pytest.mark.parametrize("groups,M,N,K", [(40, 320, 300, 96), (4, 8000, 5003, 2080)])
def test_offsets_that_descend_stay_inside_the_operands(groups, M, N, K):
    """Every second pair spans all rows, the others descend: each row of C comes from one of the groups,
    and nothing else is written (8000 rows: the walking tile; 320: 32-row tiles)."""
    print(f"mx4 descending offsets groups={groups} M={M}", flush=True)
    rng = np.random.default_rng(M)
    a, sa, va = _random_mx4(rng, (M,), K)
    b, sb, vb = _random_mx4(rng, (groups, N), K, pitch_codes=16)
    off = torch.tensor([0, M] * (groups // 2) + [0], dtype=torch.int32, device="cuda")
    out = torch.full((M + 2, N), 7.0, device="cuda")
    _ops().mx4_gemm_grouped(a, sa, b, sb, off, "f32", out=out[1:M + 1])
    assert (out[0] == 7).all() and (out[M + 1] == 7).all()
    ours = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    for e in range(groups):
        ours |= out[1:M + 1] == (va @ vb[e].t().contiguous()).float()
    assert ours.all()
    off = torch.tensor([-3, 5, 1 << 30] + [5] * (groups - 2), dtype=torch.int32, device="cuda")
    _ops().mx4_gemm_grouped(a, sa, b, sb, off, "f32", out=out[1:M + 1])
    assert (out[0] == 7).all() and (out[M + 1] == 7).all()
    assert torch.equal(out[1:6].double(), va[:5] @ vb[0].t().contiguous())
    assert torch.equal(out[6:M + 1].double(), va[5:] @ vb[1].t().contiguous())


# Sizes that take the 256×256 tile with more tiles than compute units, so that workgroups walk from
# tile to tile (test_grouped_handoff.py checks the choice): an odd pitch of C, overhang, a tail in K.
@gpu
def test_walking_tile_exact():
    M, N, K = 5100, 5003, 2080
    print(f"mx4 product M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(81)
    a, sa, va = _random_mx4(rng, (M,), K, pitch_codes=16)
    b, sb, vb = _random_mx4(rng, (N,), K)
    want = va @ vb.t().contiguous()
    for out_dtype, pad in (("f32", 1), ("bf16", 0), ("bf16", 1)):
        full = torch.full((M + 1, N + pad), -9.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().mx4_gemm(a, sa, b, sb, out_dtype, out=full[:M, :N])
        assert torch.equal(full[:M, :N], want.to(full.dtype)), out_dtype
        assert (full[M] == -9).all() and (full[:, N:] == -9).all()
    for out_dtype in ("f32", "bf16"):
        out = torch.full((M, N), 3.0, dtype=TORCH[out_dtype], device="cuda")
        _ops().mx4_gemm(a, sa, b, sb, out_dtype, out=out, alpha=0.5, beta=2.0)
        assert torch.equal(out, (0.5 * want + 6).to(out.dtype))


@gpu
def test_walking_tile_over_groups_and_replays():
    """The ragged product on the walking tile, eager and replayed with other offsets in place."""
    sizes, N, K = ([2500, 0, 1990, 257, 1253], [0, 1, 5400, 0, 599], [1200] * 5), 4603, 2080
    M, G = 6009, 5
    print(f"mx4 grouped product groups={G} M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(82)
    a, sa, va = _random_mx4(rng, (M,), K)
    b, sb, vb = _random_mx4(rng, (G, N), K)
    want, edges = [], []
    for s in sizes:
        edges.append([3] + [3 + int(v) for v in np.cumsum(s)])
        w = torch.full((M, N), 5.0, dtype=torch.float64, device="cuda")
        for e in range(G):
            w[edges[-1][e]:edges[-1][e + 1]] = va[edges[-1][e]:edges[-1][e + 1]] @ vb[e].t().contiguous()
        want.append(w)
    off = torch.tensor(edges[0], dtype=torch.int32, device="cuda")
    out = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    _ops().mx4_gemm_grouped(a, sa, b, sb, off, "bf16", out=out)
    assert torch.equal(out, want[0].to(out.dtype))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _ops().mx4_gemm_grouped(a, sa, b, sb, off, "bf16", out=out)
    for i in (1, 2, 0, 1):
        off.copy_(torch.tensor(edges[i], dtype=torch.int32))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i].to(out.dtype)), i
        eager = _ops().mx4_gemm_grouped(a, sa, b, sb, off, "f32", out=torch.full((M, N), 5.0, device="cuda"))
        assert torch.equal(eager, want[i].float()), i


@gpu
@pytest.mark.parametrize("M", [9, 600])
def test_product_offsets_past_32_bits(M):
    """Codes at nearly the largest pitch (600 rows of 8 MiB) and matrices 4 GiB apart, scales too."""
    rng, K, N = np.random.default_rng(M), 288, 40
    a, sa, va = _random_mx4(rng, (M,), K)
    b, sb, vb = _random_mx4(rng, (2, N), K)
    buf = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
    pitch = (1 << 23) - 16
    A = buf.as_strided((M, K // 2), (pitch, 1))
    A.copy_(a)
    out = _ops().mx4_gemm(A, sa, b[0], sb[0], "f32")
    assert torch.equal(out.double(), va @ vb[0].t().contiguous())
    big = buf.as_strided((2, N, K // 2), ((1 << 32) + 64, K // 2, 1))
    big.copy_(b)
    big_s = buf[1 << 20:].as_strided((2, N, K // 32), ((1 << 32) + 4096, 16, 1))
    big_s.copy_(sb)
    cut = M // 2
    off = torch.tensor([0, cut, M], dtype=torch.int32, device="cuda")
    out = _ops().mx4_gemm_grouped(a, sa, big, big_s, off, "f32")
    want = torch.cat([va[:cut] @ vb[0].t().contiguous(), va[cut:] @ vb[1].t().contiguous()])
    assert torch.equal(out.double(), want)


@gpu
def test_quantised_experts_as_a_server_runs_them():
    """Weights quantised once; each step quantises its rows and multiplies, captured and replayed with
    other rows and other offsets.  Every replay equals the eager result bit for bit, and the eager
    result the products of the decoded values within the bound of an fp32 sum."""
    ops = _ops()
    gen = torch.Generator(device="cuda").manual_seed(5)
    G, M, N, K = 6, 48, 136, 1000
    w = (torch.randn((G, N, K), generator=gen, device="cuda") * 0.05).bfloat16()
    b, sb = ops.mx4_quantize(w)
    x = torch.randn((M, K), generator=gen, device="cuda").bfloat16()
    off = torch.tensor([0, 8, 8, 20, 21, 40, 48], dtype=torch.int32, device="cuda")
    codes, scales = ops.mx4_quantize(x)
    out = torch.zeros((M, N), device="cuda")

    def step():
        ops.mx4_quantize(x, codes, scales)
        return ops.mx4_gemm_grouped(codes, scales, b, sb, off, "f32", out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    vb = ops.mx4_dequantize(b, sb, cols=K, out_dtype="f32").double()
    for edges in ([0, 8, 8, 20, 21, 40, 48], [0, 48, 48, 48, 48, 48, 48], [0, 0, 1, 2, 3, 4, 48]):
        off.copy_(torch.tensor(edges, dtype=torch.int32, device="cuda"))
        x.copy_(torch.randn((M, K), generator=gen, device="cuda").bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        out.zero_()
        assert torch.equal(got, step())
        va = ops.mx4_dequantize(codes, scales, cols=K, out_dtype="f32").double()
        for e in range(G):
            rows = slice(edges[e], edges[e + 1])
            want, mag = va[rows] @ vb[e].t().contiguous(), va[rows].abs() @ vb[e].abs().t().contiguous()
            assert ((got[rows].double() - want).abs() <= (K * 2.0 ** -23 + 2.0 ** -24) * mag).all()


@gpu
def test_torch_helper_refusals():
    ops = _ops()
    x = torch.zeros((8, 64), device="cuda")
    c, s = ops.mx4_quantize(x)
    for bad in (x.double(), x.cpu(), x.t(), x[0]):
        with pytest.raises(ValueError):
            ops.mx4_quantize(bad)
    with pytest.raises(ValueError):
        ops.mx4_quantize(x, codes=c)
    with pytest.raises(ValueError):
        ops.mx4_quantize(x, codes=c[:, :16], scales=s[:, :1])
    with pytest.raises(ValueError):
        ops.mx4_dequantize(c, s, cols=31)
    with pytest.raises(ValueError):
        ops.mx4_gemm(c, s, c, s[:, :1])
    with pytest.raises(ValueError):
        ops.mx4_gemm(c, s, c, s, out_dtype="f16")
    with pytest.raises(ValueError):
        ops.mx4_gemm(c, s, c[:, :16], s[:, :1])
    with pytest.raises(ValueError):
        ops.mx4_gemm_grouped(c, s, c, s, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(tbg.Error):
        ops.mx4_gemm(c, s.contiguous(), c, s)  # scale rows two bytes apart


@gpu
@pytest.mark.parametrize("M,edges", [
    (1000, [0, 900, 0, 900, 0, 900, 1000]),
    (2000, [0, 1900, 0, 2000]),
    (40, [0, 36, 0, 36, 0, 40]),
    (3000, [0, 2990] * 100 + [0, 3000]),
    (6000, [5, 5900, 0, 5900, 0, 6000]),
])
def test_rows_of_descending_offsets_belong_to_the_first_group_that_reaches_them(M, edges):
    """An offset below an earlier one counts as that one, so every row up to the largest offset has one
    group, and none is left out (groups that claim more tiles than ascending ones can make)."""
    print(f"mx4 descending offsets M={M} groups={len(edges) - 1}", flush=True)
    rng, G, K = np.random.default_rng(M), len(edges) - 1, 96
    good = np.maximum.accumulate(edges).tolist()
    a, sa, va = _random_mx4(rng, (M,), K)
    for N in (40, 3000 if M > 5000 else 500):
        b, sb, vb = _random_mx4(rng, (G, N), K)
        out = torch.full((M + 2, N), 7.0, device="cuda")
        _ops().mx4_gemm_grouped(a, sa, b, sb, torch.tensor(edges, dtype=torch.int32, device="cuda"), "f32",
                                out=out[1:M + 1])
        want = torch.full((M + 2, N), 7.0, device="cuda")
        for e in range(G):
            lo, hi = good[e], good[e + 1]
            if lo < hi:
                want[1 + lo:1 + hi] = (va[lo:hi] @ vb[e].t().contiguous()).float()
        assert torch.equal(out, want), N


@gpu
def test_rows_without_a_column():
    """K == 0 from end to end: no codes, no scales, and the empty sum."""
    ops = _ops()
    x, w = torch.zeros((5, 0), device="cuda"), torch.zeros((2, 7, 0), device="cuda")
    (a, sa), (b, sb) = ops.mx4_quantize(x), ops.mx4_quantize(w)
    assert ops.mx4_dequantize(a, sa, cols=0).shape == (5, 0)
    out = ops.mx4_gemm(a, sa, b[0], sb[0], "f32", out=torch.full((5, 7), float("nan"), device="cuda"))
    assert (out == 0).all()
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    out = ops.mx4_gemm_grouped(a, sa, b, sb, off, "f32", out=torch.full((5, 7), 3.0, device="cuda"), beta=2.0)
    assert (out[:4] == 6).all() and (out[4] == 3).all()


def _all_codes():
    """Every code under every scale byte: codes (256, 16 bytes), scale bytes (256, 1), the values."""
    code = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 1))
    scale = np.arange(256, dtype=np.uint8)[:, None]
    held = np.zeros((256, 16), dtype=np.uint8)
    held[:, :1] = scale
    return torch.from_numpy(pack(code)).cuda(), torch.from_numpy(held).cuda()[:, :1], ref_values(code, scale)


@gpu
@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
def test_every_code_under_every_scale_decodes_to_the_value_rounded_once(out_dtype):
    """The format's ends included: subnormal values of fp32, bf16 and fp16, values that fp16 rounds (to a
    subnormal, to zero with its sign) and those past its largest (infinity, as rounding gives)."""
    codes, scales, want = _all_codes()
    got = _ops().mx4_dequantize(codes, scales, out_dtype=out_dtype).cpu()
    assert got[255].isnan().all()
    # (two significant bits: fp32 and bf16 hold every value below 2^128 exactly)
    with np.errstate(over="ignore"):
        w = torch.from_numpy(want[:255].astype(np.float16 if out_dtype == "f16" else np.float32)).to(TORCH[out_dtype])
    bits = torch.int32 if out_dtype == "f32" else torch.int16
    bad = (got[:255].view(bits) != w.view(bits)).nonzero()
    assert len(bad) == 0, [(int(r), int(c), got[r, c].item(), w[r, c].item()) for r, c in bad[:8]]


# one size for each kernel of the product (test_grouped_handoff.py checks the choice for such sizes)
ENDS = [(3, 300, 2080), (20, 300, 2080), (70, 300, 2080), (2000, 2000, 2080), (4000, 4000, 4128)]


@gpu
@pytest.mark.parametrize("M,N,K", ENDS)
def test_product_of_scales_at_the_ends_of_the_format(M, N, K):
    """Scales from 2^-127 to 2^127 that cancel block by block: every term is a multiple of 1/4 of at most
    36, so the sum is exact (144·K quarters < 2^24)."""
    print(f"mx4 product at the format's ends M={M} N={N} K={K}", flush=True)
    rng = np.random.default_rng(M)
    a, sa, _ = _random_mx4(rng, (M,), K, spread=0)
    b, sb, _ = _random_mx4(rng, (N,), K, spread=0)
    e = rng.integers(0, 255, K // 32)
    e[:8] = [0, 254, 1, 253, 2, 252, 127, 128]
    ca, cb = a.cpu().numpy(), b.cpu().numpy()
    one = np.full(K // 32, 127, dtype=np.uint8)
    va = torch.from_numpy(ref_values(unpack(ca), np.broadcast_to(one, (M, K // 32)))).cuda()
    vb = torch.from_numpy(ref_values(unpack(cb), np.broadcast_to(one, (N, K // 32)))).cuda()
    sa.copy_(torch.from_numpy(e.astype(np.uint8)).expand(M, -1))
    sb.copy_(torch.from_numpy((254 - e).astype(np.uint8)).expand(N, -1))
    want = va @ vb.t().contiguous()
    for out_dtype in ("f32", "bf16"):
        out = _ops().mx4_gemm(a, sa, b, sb, out_dtype)
        assert torch.equal(out, want.to(out.dtype)), out_dtype
