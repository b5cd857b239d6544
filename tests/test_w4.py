"""Products with weights in 4-bit codes and group scales (tbg_w4_gemm, tbg_w4_gemm_grouped) against the
definition in 64 bits.

Small whole activations and scales that are powers of two have sums that fp32 holds exactly, so there the
output must equal the reference rounded once to C's type, bit for bit.  Real operands are held to the bound of
the kernel's sums: per group an fp32 sum of G exact products a·c (and one of a alone, times z, for bf16), then
two fused steps with the scale, then the groups' and the waves' sums; every step is off by at most one
unit in the last place (2^-23) of the magnitudes so far, so with mag = sum |a|·|s|·(c + z)
|C - exact| <= (K + 3·K/G + 16)·2^-23·mag + eps/2·(|exact| + that)."""
import numpy as np
import pytest
import torch

import tiled_bf16_gemm_amd as tbg

gpu = pytest.mark.gpu
PTR = 0x7F00_0000_0000  # a device-like address: argument checks never touch memory
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _ops():
    from tiled_bf16_gemm_amd import torch_ops
    return torch_ops


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# ---- refusals (CPU) -------------------------------------------------------------------------------

def _args(**over):
    a = dict(M=4, N=16, K=128, group=32, alpha=1.0, A=PTR, lda=128, ab_dtype="bf16", codes=PTR, ldb=64, scales=PTR,
             ld_s=16, zeros=PTR, ld_z=16, beta=0.0, C=PTR, ldc=16, c_dtype="bf16")
    a.update(over)
    return a


DENSE = [
    (dict(M=-1), tbg.ERR_INVALID_VALUE),
    (dict(N=-1), tbg.ERR_INVALID_VALUE),
    (dict(K=-32), tbg.ERR_INVALID_VALUE),
    (dict(M=(1 << 30) + 1), tbg.ERR_UNSUPPORTED),
    (dict(N=(1 << 30) + 1, ld_s=1 << 31, ld_z=1 << 31, ldc=1 << 31), tbg.ERR_UNSUPPORTED),
    (dict(group=16), tbg.ERR_INVALID_VALUE),
    (dict(group=0), tbg.ERR_INVALID_VALUE),
    (dict(group=256, K=256, lda=256, ldb=128), tbg.ERR_INVALID_VALUE),
    (dict(K=96, group=64), tbg.ERR_INVALID_VALUE),
    (dict(K=130), tbg.ERR_INVALID_VALUE),
    (dict(ab_dtype="f32"), tbg.ERR_INVALID_VALUE),
    (dict(c_dtype="f16"), tbg.ERR_INVALID_VALUE),
    (dict(A=0), tbg.ERR_INVALID_VALUE),
    (dict(A=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(codes=0), tbg.ERR_INVALID_VALUE),
    (dict(codes=PTR + 8), tbg.ERR_MISALIGNED),
    (dict(ldb=72), tbg.ERR_MISALIGNED),
    (dict(ldb=48), tbg.ERR_INVALID_VALUE),
    (dict(ldb=1 << 23), tbg.ERR_UNSUPPORTED),
    (dict(scales=0), tbg.ERR_INVALID_VALUE),
    (dict(scales=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(ld_s=15), tbg.ERR_INVALID_VALUE),
    (dict(ld_s=(1 << 28) + 1), tbg.ERR_UNSUPPORTED),
    (dict(ld_z=(1 << 28) + 1), tbg.ERR_UNSUPPORTED),
    (dict(ld_z=15), tbg.ERR_INVALID_VALUE),
    (dict(lda=127), tbg.ERR_INVALID_VALUE),
    (dict(ldc=15), tbg.ERR_INVALID_VALUE),
    (dict(C=0), tbg.ERR_INVALID_VALUE),
    (dict(C=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(M=1 << 30, N=1 << 30, ld_s=1 << 30, ld_z=1 << 30, ldc=1 << 30), (tbg.ERR_UNSUPPORTED, tbg.ERR_NO_DEVICE)),
]


@pytest.mark.parametrize("over,status", DENSE)
def test_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.w4_gemm(**_args(**over))
    assert e.value.status in (status if isinstance(status, tuple) else (status,)), e.value


def _grouped_args(**over):
    a = dict(groups=2, M=4, N=16, K=128, group=32, offsets=PTR, source=PTR, a_rows=4, top_k=2, alpha=1.0, A=PTR, lda=128,
             ab_dtype="bf16", codes=PTR, ldb=64, stride_b=16 * 64, scales=PTR, ld_s=16, stride_s=64, zeros=PTR, ld_z=16,
             stride_z=64, beta=0.0, C=PTR, ldc=16, c_dtype="bf16")
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(groups=-1), tbg.ERR_INVALID_VALUE),
    (dict(groups=4097), tbg.ERR_UNSUPPORTED),
    (dict(offsets=0), tbg.ERR_INVALID_VALUE),
    (dict(offsets=PTR + 2), tbg.ERR_MISALIGNED),
    (dict(source=PTR + 2), tbg.ERR_MISALIGNED),
    (dict(a_rows=-1), tbg.ERR_INVALID_VALUE),
    (dict(a_rows=0), tbg.ERR_INVALID_VALUE),
    (dict(a_rows=(1 << 30) + 1), tbg.ERR_UNSUPPORTED),
    (dict(top_k=0), tbg.ERR_INVALID_VALUE),
    (dict(top_k=(1 << 30) + 1), tbg.ERR_UNSUPPORTED),
    (dict(stride_b=16 * 64 - 16), tbg.ERR_INVALID_VALUE),
    (dict(stride_b=16 * 64 + 8), tbg.ERR_MISALIGNED),
    (dict(stride_s=63), tbg.ERR_INVALID_VALUE),
    (dict(stride_z=63), tbg.ERR_INVALID_VALUE),
    (dict(group=48), tbg.ERR_INVALID_VALUE),
])
def test_grouped_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.w4_gemm_grouped(**_grouped_args(**over))
    assert e.value.status == status, e.value


def test_no_ops_need_no_device():
    tbg.w4_gemm(**_args(M=0))
    tbg.w4_gemm(**_args(N=0, ldc=1))
    tbg.w4_gemm_grouped(**_grouped_args(groups=0, offsets=0))
    tbg.w4_gemm_grouped(**_grouped_args(M=0))


def test_unused_pitches_do_not_limit_columns():
    """alpha 0 leaves A and W out, their pitches with them: N past the limit of a pitch of codes is taken."""
    N = (1 << 23) + 32
    tbg.w4_gemm(**_args(M=0, N=N, alpha=0.0, lda=0, ldb=0, ld_s=0, ld_z=0, ldc=N))


@gpu
def test_alpha_zero_of_many_columns():
    N = (1 << 23) + 17
    c = torch.ones(N, device="cuda")
    tbg.w4_gemm(**_args(M=1, N=N, alpha=0.0, A=0, codes=0, scales=0, zeros=0, beta=2.0, C=c.data_ptr(), ldc=N,
                        c_dtype="f32"), stream=torch.cuda.current_stream().cuda_stream)
    assert bool((c == 2).all())


def test_helpers_refuse_host_tensors():
    a, c, s = torch.zeros((2, 64)).half(), torch.zeros((8, 32), dtype=torch.uint8), torch.zeros((2, 8)).half()
    with pytest.raises(ValueError):
        _ops().w4_gemm(a, c, s)
    with pytest.raises(ValueError):
        _ops().w4_gemm_grouped(a, c[None], s[None], torch.zeros(2, dtype=torch.int32))


# ---- operands and the definition ------------------------------------------------------------------

def _pack(code):
    """Codes 0..15 (…, N, K) two to a byte, the lower nibble first, rows at 16 bytes."""
    K = code.shape[-1]
    pitch = -(-K // 32) * 16
    full = torch.zeros((*code.shape[:-1], pitch), dtype=torch.uint8, device=code.device)
    full[..., :K // 2] = code[..., 0::2] | (code[..., 1::2] << 4)
    return full[..., :K // 2]


def _operands(gen, lead, N, K, G, dtype, zeros, whole):
    """code, scales, zeros (or None) of matrices `lead` + (N, K)."""
    code = torch.randint(0, 16, (*lead, N, K), device="cuda", generator=gen, dtype=torch.uint8)
    if whole:
        s = 2.0 ** torch.randint(-2, 2, (*lead, K // G, N), device="cuda", generator=gen).float()
        s = s * (1 - 2 * torch.randint(0, 2, s.shape, device="cuda", generator=gen)).float()
    else:
        s = 0.01 * torch.rand((*lead, K // G, N), device="cuda", generator=gen) + 0.001
    z = torch.randint(0, 16, s.shape, device="cuda", generator=gen, dtype=torch.uint8) if zeros else None
    return code, s.to(TORCH[dtype]), z


def _weights(code, s, z, plus=False):
    """W in 64 bits; plus: |s|·(c + z) instead."""
    G = code.shape[-1] // s.shape[-2] if s.shape[-2] else 1
    s = s.double().transpose(-1, -2).repeat_interleave(G, -1)
    zero = torch.full_like(s, 8.0) if z is None else z.double().transpose(-1, -2).repeat_interleave(G, -1)
    return s.abs() * (code.double() + zero) if plus else s * (code.double() - zero)


def _bound(a, code, s, z, exact, out):
    K, parts = code.shape[-1], s.shape[-2]
    acc = (K + 3 * parts + 16) * 2.0 ** -23 * (a.double().abs() @ _weights(code, s, z, True).t().contiguous())
    sub = 2.0 ** -25 if out == "f16" else 0.0
    return acc + torch.finfo(TORCH[out]).eps / 2 * (exact.abs() + acc) + sub


SHAPES = [(1, 1, 32, 32), (1, 16, 128, 128), (3, 17, 96, 32), (16, 64, 256, 64), (5, 100, 192, 64), (17, 33, 640, 128),
          (33, 257, 544, 32), (64, 48, 1152, 128), (65, 130, 2048, 64), (130, 20, 4096, 128), (2, 5000, 160, 32),
          (20, 9000, 128, 128), (40, 9001, 64, 64), (7, 15, 8192, 32), (40, 16400, 160, 32), (200, 6200, 192, 64),
          (100, 12300, 384, 128)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,G", SHAPES)
def test_whole_numbers_are_exact(M, N, K, G, dtype):
    ops = _ops()
    for zeros in (False, True):
        print(f"w4 {M}x{N}x{K} group {G} {dtype} zeros {zeros}", flush=True)
        g = _gen(M + N + K)
        code, s, z = _operands(g, (), N, K, G, dtype, zeros, True)
        a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).to(TORCH[dtype])
        exact = a.double() @ _weights(code, s, z).t().contiguous()  # below 4·15·8192·2 = 2^20, in quarters
        for out in ("f32", dtype):
            full = torch.full((M + 2, N + 3), 9.0, dtype=TORCH[out], device="cuda")
            got = ops.w4_gemm(a, _pack(code), s, z, out_dtype=out, out=full[1:-1, :N])
            want = exact.float().to(TORCH[out])
            assert torch.equal(got, want), float((got.double() - exact).abs().max())
            assert bool((full[0] == 9).all()) and bool((full[-1] == 9).all()) and bool((full[:, N:] == 9).all())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,G", SHAPES)
def test_within_the_bound_of_its_sums(M, N, K, G, dtype):
    ops = _ops()
    for zeros, out in ((False, "f32"), (True, dtype), (True, "f32")):
        print(f"w4 {M}x{N}x{K} group {G} {dtype} zeros {zeros} out {out}", flush=True)
        g = _gen(M + N + K + 1)
        code, s, z = _operands(g, (), N, K, G, dtype, zeros, False)
        a = (torch.randn((M, K), device="cuda", generator=g) + 0.5).to(TORCH[dtype])
        exact = a.double() @ _weights(code, s, z).t().contiguous()
        got = ops.w4_gemm(a, _pack(code), s, z, out_dtype=out)
        assert bool(((got.double() - exact).abs() <= _bound(a, code, s, z, exact, out)).all())


@gpu
def test_every_code_and_zero():
    """Every code against every zero byte, 0 to 255, of a single 1 in A: W itself comes out."""
    ops = _ops()
    for dtype in ("bf16", "f16"):
        K, N = 32, 256
        code = (torch.arange(K, device="cuda", dtype=torch.int32) % 16).to(torch.uint8).expand(N, K).contiguous()
        z = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8)[None].contiguous()
        s = torch.full((1, N), 0.5, device="cuda", dtype=TORCH[dtype])
        a = torch.eye(K, device="cuda", dtype=TORCH[dtype])
        got = ops.w4_gemm(a, _pack(code), s, z, out_dtype="f32")
        assert torch.equal(got.double(), _weights(code, s, z).t())


@gpu
def test_order_of_the_codes():
    """Each k alone, over whole blocks of 128 and a part of one, against random codes."""
    ops = _ops()
    for dtype in ("bf16", "f16"):
        for G in (32, 64, 128):
            K, N = 3 * 128 + (G if G < 128 else 0), 48
            code, s, z = _operands(_gen(G), (), N, K, G, dtype, True, True)
            a = torch.eye(K, device="cuda", dtype=TORCH[dtype])
            got = ops.w4_gemm(a, _pack(code), s, z, out_dtype="f32")
            assert torch.equal(got.double(), _weights(code, s, z).t())


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(5, 32800), (30, 32800), (60, 32800), (9, 400), (9, 7000), (9, 12400)])
def test_every_number_of_blocks(M, N, dtype):
    """Each kernel over sums of less than one block of 128 up to nine, whole or not."""
    ops = _ops()
    for K, G in ((32, 32), (96, 32), (128, 128), (160, 32), (192, 64), (256, 128), (352, 32), (384, 64), (512, 128), (640, 64),
                 (672, 32), (768, 128), (1088, 64), (1152, 32)):
        print(f"w4 {M}x{N}x{K} group {G} {dtype}", flush=True)
        code, s, z = _operands(_gen(K), (), N, K, G, dtype, K % 64 == 0, True)
        a = torch.randint(-4, 5, (M, K), device="cuda", generator=_gen(K + 1)).to(TORCH[dtype])
        want = (a.double() @ _weights(code, s, z).t().contiguous()).float()
        assert torch.equal(ops.w4_gemm(a, _pack(code), s, z, out_dtype="f32"), want)


@gpu
@pytest.mark.parametrize("M,N,K", [(40, 70, 512), (40, 32800, 256), (30, 32800, 160), (16, 32800, 96), (16, 12400, 160)])
def test_infinities_and_huge_values(M, N, K):
    """Rows that hold an infinity, a NaN or values near the end of bf16's range come out as the definition's sum, and
    the others are not touched by them."""
    ops = _ops()
    g = _gen(4)
    G, inf, big = 32, float("inf"), 2.0 ** 127
    code, s, z = _operands(g, (), N, K, G, "bf16", True, True)
    for dtype in ("bf16", "f16"):
        sc = s.to(TORCH[dtype])
        a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).to(TORCH[dtype])
        a[3, 17], a[9, 70], a[11, 5] = inf, -inf, float("nan")
        if dtype == "bf16":
            a[14, 40], a[14, 41] = big, -big  # c·a passes fp32's range, (c - z)·a or the sum need not
        w = _weights(code, sc, z)
        rest = [r for r in range(M) if r not in (3, 9, 11, 14)]
        exact = a[rest].double() @ w.t().contiguous()
        got = ops.w4_gemm(a, _pack(code), sc, z, out_dtype="f32")
        # rows of infinities: inf·0 is NaN, the others infinite with the weight's sign
        for r, k, sign in ((3, 17, 1.0), (9, 70, -1.0)):
            want = torch.where(w[:, k] == 0, float("nan"), sign * w[:, k].sign() * inf)
            assert torch.equal(torch.nan_to_num(got[r].double(), nan=7.0), torch.nan_to_num(want, nan=7.0))
        assert bool(torch.isnan(got[11]).all())
        assert torch.equal(got[rest].double(), exact)
        if dtype == "bf16":
            cz = code.double() - z.double().t().repeat_interleave(G, -1)
            fits = (cz[:, 40].abs() <= 1) & (cz[:, 41].abs() <= 1)
            assert bool(torch.isfinite(got[14][fits & (cz[:, 40] == cz[:, 41])]).all())


@gpu
def test_strides_and_alignment():
    """A at any element, pitches of codes, scales and zeros, a transposed stack's strides."""
    ops = _ops()
    g = _gen(6)
    M, N, K, G = 9, 50, 256, 64
    for dtype in ("bf16", "f16"):
        code, s, z = _operands(g, (), N, K, G, dtype, True, True)
        a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).to(TORCH[dtype])
        want = (a.double() @ _weights(code, s, z).t().contiguous()).float()
        for first, ld in ((0, K), (1, K + 1), (3, K + 7), (5, 2 * K)):
            flat = torch.full((first + M * ld,), float("nan"), device="cuda", dtype=TORCH[dtype])
            view = flat[first:].as_strided((M, K), (ld, 1), first)
            view.copy_(a)
            codes = torch.full((N, K // 2 + 16 * first), 0xFF, dtype=torch.uint8, device="cuda")[:, :K // 2]
            codes.copy_(_pack(code))
            sc = torch.full((K // G, N + first), float("nan"), dtype=TORCH[dtype], device="cuda")[:, :N]
            sc.copy_(s)
            ze = torch.full((K // G, N + 2 * first), 255, dtype=torch.uint8, device="cuda")[:, :N]
            ze.copy_(z)
            assert torch.equal(ops.w4_gemm(view, codes, sc, ze, out_dtype="f32"), want)
        one = a.expand(4, M, K)[:, 2]  # one row four times: a pitch of 0 below the row is refused
        with pytest.raises(tbg.Error):
            ops.w4_gemm(one, _pack(code), s, z, out_dtype="f32")
        assert torch.equal(ops.w4_gemm(a[2:3], _pack(code), s, z, out_dtype="f32"), want[2:3])


@gpu
def test_alpha_and_beta():
    ops = _ops()
    g = _gen(7)
    M, N, K, G = 20, 40, 256, 32
    code, s, z = _operands(g, (), N, K, G, "bf16", True, True)
    a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).bfloat16()
    exact = a.double() @ _weights(code, s, z).t().contiguous()
    old = torch.randint(-8, 9, (M, N), device="cuda", generator=g).float()
    for out in ("f32", "bf16"):
        for alpha, beta in ((0.5, 1.0), (-1.0, 0.0), (0.0, 0.5), (0.0, 0.0), (2.0, -0.25)):
            c = old.to(TORCH[out], copy=True)
            got = ops.w4_gemm(a, _pack(code), s, z, out_dtype=out, out=c, alpha=alpha, beta=beta)
            assert torch.equal(got, (alpha * exact + beta * old.double()).float().to(TORCH[out]))
    nan = torch.full((M, N), float("nan"), device="cuda")
    assert torch.equal(ops.w4_gemm(a, _pack(code), s, z, out_dtype="f32", out=nan.clone(), beta=0.0), exact.float())
    assert bool((ops.w4_gemm(a * float("nan"), _pack(code), s, z, out_dtype="f32", alpha=0.0) == 0).all())
    with pytest.raises(ValueError):
        ops.w4_gemm(a, _pack(code), s, z, beta=1.0)


@gpu
def test_no_sum():
    """K = 0: beta·C, zeros without."""
    ops = _ops()
    a = torch.zeros((3, 0), device="cuda").bfloat16()
    codes, s = torch.zeros((5, 0), dtype=torch.uint8, device="cuda"), torch.zeros((0, 5), device="cuda").bfloat16()
    assert bool((ops.w4_gemm(a, codes, s) == 0).all())
    c = torch.full((3, 5), 3.0, device="cuda").bfloat16()
    assert bool((ops.w4_gemm(a, codes, s, out=c, beta=2.0) == 6).all())
    assert ops.w4_gemm(torch.zeros((0, 64), device="cuda").half(), torch.zeros((5, 32), dtype=torch.uint8, device="cuda"),
                       torch.zeros((1, 5), device="cuda").half(), out_dtype="f16").shape == (0, 5)


# ---- ragged groups --------------------------------------------------------------------------------

SPLITS = [([1], 16, 128, 128), ([0, 3, 0, 1, 5], 40, 192, 64), ([2, 1, 1, 0, 4, 1, 1, 2], 2048, 256, 128),
          ([17, 0, 31, 16], 100, 320, 32), ([64, 65, 1, 0, 200], 130, 256, 64), ([0, 0, 0], 16, 64, 32),
          ([3] * 100, 33, 96, 32), ([1] * 70, 700, 128, 64),
          ([40, 1, 90, 33, 0, 70, 64, 22], 2900, 160, 32), ([20, 1, 33, 0, 32, 17, 16, 40] * 2, 2050, 640, 64)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("sizes,N,K,G", SPLITS)
def test_ragged_groups_are_exact(sizes, N, K, G, dtype):
    ops = _ops()
    for first, tail, zeros in ((0, 0, True), (3, 7, False)):
        print(f"w4 grouped {len(sizes)} groups, {sum(sizes)} rows, {N}x{K} group {G} {dtype} first {first}", flush=True)
        edges = [first] + [first + int(v) for v in np.cumsum(sizes)]
        M, E = edges[-1] + tail, len(sizes)
        g = _gen(N + K + first)
        code, s, z = _operands(g, (E,), N, K, G, dtype, zeros, True)
        off = torch.tensor(edges, dtype=torch.int32, device="cuda")
        top_k = 3
        T = M // top_k + 1
        tokens = torch.randint(-4, 5, (T, K), device="cuda", generator=g).to(TORCH[dtype])
        source = torch.randperm(T * top_k, device="cuda", generator=g)[:M].to(torch.int32)
        rows = tokens[(source // top_k).long()]
        for out in ("f32", dtype):
            want = torch.full((M, N), 9.0, dtype=TORCH[out], device="cuda")
            for e in range(E):
                r = slice(edges[e], edges[e + 1])
                w = _weights(code[e], s[e], None if z is None else z[e])
                want[r] = (rows[r].double() @ w.t().contiguous()).float().to(TORCH[out])
            for a, src in ((rows, None), (tokens, source)):
                got = ops.w4_gemm_grouped(a, _pack(code), s, off, z, source=src, top_k=top_k, out_dtype=out,
                                          out=torch.full((M, N), 9.0, dtype=TORCH[out], device="cuda"))
                assert torch.equal(got, want)


@gpu
def test_sources_and_offsets_outside_are_the_nearest():
    ops = _ops()
    g = _gen(5)
    E, N, K, G, M, T, k = 3, 32, 128, 64, 12, 4, 2
    code, s, z = _operands(g, (E,), N, K, G, "bf16", True, True)
    tokens = torch.randint(-4, 5, (T, K), device="cuda", generator=g).bfloat16()
    source = torch.tensor([0, 1, 2, -1, -2 ** 31, 8, 9, 2 ** 31 - 1, 3, 4, 5, 7], dtype=torch.int32, device="cuda")
    row = (source.long().clamp(min=0) // k).clamp(max=T - 1)
    off = torch.tensor([-5, 4, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    got = ops.w4_gemm_grouped(tokens, _pack(code), s, off, z, source=source, top_k=k, out_dtype="f32",
                              out=torch.full((M, N), 9.0, device="cuda"))
    # rows 0..3 group 0, group 1 empty (its end lies before), rows 4..11 group 2
    for e, r in ((0, slice(0, 4)), (2, slice(4, 12))):
        assert torch.equal(got[r], (tokens[row[r]].double() @ _weights(code[e], s[e], z[e]).t().contiguous()).float())


@gpu
def test_codes_past_4_gib():
    """A stack whose last matrix lies past 2^32 bytes."""
    ops = _ops()
    E, N, K, G = 3, 16, 128, 128
    code, s, z = _operands(_gen(2), (E,), N, K, G, "bf16", False, True)
    stride = (5 << 30) // 2 // 16 * 16
    flat = torch.empty(2 * stride + N * K // 2, dtype=torch.uint8, device="cuda")
    codes = flat.as_strided((E, N, K // 2), (stride, K // 2, 1))
    codes.copy_(_pack(code))
    a = torch.randint(-4, 5, (6, K), device="cuda").bfloat16()
    off = torch.tensor([0, 2, 4, 6], dtype=torch.int32, device="cuda")
    got = ops.w4_gemm_grouped(a, codes, s, off, out_dtype="f32")
    for e in range(E):
        r = slice(2 * e, 2 * e + 2)
        assert torch.equal(got[r], (a[r].double() @ _weights(code[e], s[e], None).t().contiguous()).float())


@gpu
def test_captured_product_replays_with_other_rows():
    ops = _ops()
    g = _gen(8)
    E, N, K, G, T, k = 16, 96, 256, 128, 8, 2
    code, s, z = _operands(g, (E,), N, K, G, "bf16", True, True)
    codes = _pack(code)
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    x = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((T * k, N), device="cuda")

    def step():
        off, src, place = ops.expert_sort(ids, E)
        ops.w4_gemm_grouped(x, codes, s, off, z, source=src, top_k=k, out_dtype="f32", out=out)
        return ops.expert_combine(out, place)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    w = torch.stack([_weights(code[e], s[e], z[e]) for e in range(E)])
    for i in range(4):
        ids.copy_(torch.randint(0, E, (T, k), device="cuda", generator=g))
        x.copy_(torch.randint(-4, 5, (T, K), device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.stack([sum(w[int(e)] @ x[t].double() for e in ids[t]) for t in range(T)])
        assert torch.equal(held.double(), want), i
        assert torch.equal(step(), held)


@gpu
def test_on_another_stream():
    ops = _ops()
    g = _gen(3)
    code, s, z = _operands(g, (), 300, 512, 32, "f16", True, True)
    a = torch.randint(-4, 5, (5, 512), device="cuda", generator=g).half()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = ops.w4_gemm(a, _pack(code), s, z, out_dtype="f32", stream=st)
    st.synchronize()
    assert torch.equal(got.double(), a.double() @ _weights(code, s, z).t().contiguous())


@gpu
def test_helpers_refuse_on_the_device():
    ops = _ops()
    a = torch.zeros((4, 128), device="cuda").half()
    c = torch.zeros((8, 64), dtype=torch.uint8, device="cuda")
    s = torch.zeros((4, 8), device="cuda").half()
    z = torch.zeros((4, 8), dtype=torch.uint8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    st = [t.expand(2, *t.shape).contiguous() for t in (c, s, z)]
    for call in (lambda: ops.w4_gemm(a.float(), c, s), lambda: ops.w4_gemm(a, c.char(), s), lambda: ops.w4_gemm(a, c, s.bfloat16()),
                 lambda: ops.w4_gemm(a, c, s[:, :7]), lambda: ops.w4_gemm(a, c, s[:3]), lambda: ops.w4_gemm(a[:, :96], c, s),
                 lambda: ops.w4_gemm(a, c, s, z[:3]), lambda: ops.w4_gemm(a, c, s, z.char()), lambda: ops.w4_gemm(a, c, s, out_dtype="bf16"),
                 lambda: ops.w4_gemm(a, c, s, out_dtype="f16", out=a), lambda: ops.w4_gemm(a, c, s.cpu()), lambda: ops.w4_gemm(a, c, s, z.cpu()),
                 lambda: ops.w4_gemm(a, c.t(), s),
                 lambda: ops.w4_gemm_grouped(a, c, s, off), lambda: ops.w4_gemm_grouped(a, st[0], st[1], off[:2]),
                 lambda: ops.w4_gemm_grouped(a, st[0], st[1][:1], off), lambda: ops.w4_gemm_grouped(a, st[0], st[1], off.long()),
                 lambda: ops.w4_gemm_grouped(a, st[0], st[1], off, source=off.long()),
                 lambda: ops.w4_gemm_grouped(a, st[0], st[1], off, st[2][:, :3])):
        with pytest.raises(ValueError):
            call()


# ---- together -------------------------------------------------------------------------------------

@gpu
def test_decoding_step_of_a_layer_of_experts():
    """A server's step: sort, up and gate products that read the tokens through the sort, the elementwise product
    in between, the down product, combine; whole numbers and power-of-two scales, so all of it is exact."""
    ops = _ops()
    g = _gen(12)
    T, k, E, H, F, G = 8, 4, 32, 128, 256, 64
    ids = torch.argsort(torch.rand((T, E), device="cuda", generator=g), dim=1)[:, :k].to(torch.int32).contiguous()
    ids[T - 1] = -1
    x = torch.randint(-1, 2, (T, H), device="cuda", generator=g).bfloat16()

    def matrix(N, K):
        code = torch.randint(7, 10, (E, N, K), device="cuda", generator=g, dtype=torch.uint8)
        s = 2.0 ** torch.randint(-1, 2, (E, K // G, N), device="cuda", generator=g).float()
        return code, s.bfloat16()

    up, down = matrix(F, H), matrix(H, F)
    w = torch.randint(1, 5, (T, k), device="cuda", generator=g).float() / 4
    off, src, place = ops.expert_sort(ids, E)
    h = ops.w4_gemm_grouped(x, _pack(up[0]), up[1], off, source=src, top_k=k, out_dtype="f32",
                            out=torch.zeros((T * k, F), device="cuda"))
    a = h.clamp(-8, 8).round().bfloat16()  # whole numbers of few bits again
    y = ops.w4_gemm_grouped(a, _pack(down[0]), down[1], off, out_dtype="f32", out=torch.zeros((T * k, H), device="cuda"))
    out = ops.expert_combine(y, place, w)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for t in range(T - 1):
        for j in range(k):
            e = int(ids[t, j])
            hh = (_weights(up[0][e], up[1][e], None) @ x[t].double()).clamp(-8, 8).round()
            want[t] += float(w[t, j]) * (_weights(down[0][e], down[1][e], None) @ hh)
    assert torch.equal(out.double(), want)


# ---- rows beside one that is not finite -------------------------------------------------------------

# every kernel and tile: K split over the waves with 16, 32 and 64 columns, panels of 16, 32 and 64 rows
KERNELS = [(9, 400), (9, 7000), (9, 12400), (16, 32800), (30, 32800), (60, 32800)]


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", KERNELS)
def test_rows_keep_their_bits_beside_others_that_are_not_finite(M, N, dtype):
    """A row's value, to the last bit, does not depend on what another row of its tile holds: a NaN or an infinity
    there (another request's, a padding row's) leaves it as it is.  Real operands: another order of the sums shows."""
    ops = _ops()
    for K, G, zeros, out, beta in ((544, 32, True, "f32", 0.0), (256, 128, False, dtype, 0.0), (192, 64, True, "f32", -0.75)):
        print(f"w4 {M}x{N}x{K} group {G} {dtype} beside a row that is not finite, beta {beta}", flush=True)
        g = _gen(M + N + K)
        code, s, z = _operands(g, (), N, K, G, dtype, zeros, False)
        codes = _pack(code)
        a = torch.randn((M, K), device="cuda", generator=g).to(TORCH[dtype])
        old = torch.randn((M, N), device="cuda", generator=g).to(TORCH[out])
        want = ops.w4_gemm(a, codes, s, z, out_dtype=out, out=old.clone(), beta=beta)
        a[3, 17], a[5, 70], a[M - 1, K - 1] = float("inf"), float("nan"), float("-inf")
        got = ops.w4_gemm(a, codes, s, z, out_dtype=out, out=old.clone(), beta=beta)
        rest = [r for r in range(M) if r not in (3, 5, M - 1)]
        assert torch.equal(got[rest], want[rest]), float((got[rest].double() - want[rest].double()).abs().max())
        assert bool(torch.isfinite(want).all()) and not bool(torch.isfinite(got[[3, 5, M - 1]]).any())


@gpu
def test_rows_of_groups_keep_their_bits_beside_others_that_are_not_finite():
    """The same over ragged groups, whose rows read A through source: also where a token that is not finite is the
    last row of its group, which the rows past its end repeat."""
    ops = _ops()
    for sizes, N in (([5, 0, 1, 17, 9], 700), ([40, 33, 64, 1, 90], 7000)):
        E, M, K, G = len(sizes), sum(sizes), 320, 64
        g = _gen(N)
        code, s, z = _operands(g, (E,), N, K, G, "bf16", True, False)
        codes = _pack(code)
        off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")
        a = torch.randn((M, K), device="cuda", generator=g).bfloat16()
        source = torch.randperm(M, device="cuda", generator=g).to(torch.int32)
        want = ops.w4_gemm_grouped(a, codes, s, off, z, source=source, out_dtype="f32")
        bad = [0, sizes[0] - 1, M - 1]
        a[source[bad].long(), 33] = float("inf")
        got = ops.w4_gemm_grouped(a, codes, s, off, z, source=source, out_dtype="f32")
        rest = [r for r in range(M) if r not in bad]
        assert torch.equal(got[rest], want[rest])
        assert bool(torch.isfinite(want).all()) and not bool(torch.isfinite(got[bad]).any())


@gpu
@pytest.mark.parametrize("M,N", KERNELS)
def test_values_near_the_end_of_the_range(M, N):
    """c·a passes fp32's range where (c - z)·a does not: such an element is the definition's sum, off by the bound of
    a sum of a·(c - z) itself, whose terms with c = z are nothing at all; C's old value is read once for it."""
    ops = _ops()
    K, G, row, at, big = 544, 32, 6, 77, 1.5 * 2.0 ** 126
    g = _gen(M + N)
    code, s, z = _operands(g, (), N, K, G, "bf16", True, True)
    z[at // G] = torch.randint(5, 15, (N,), device="cuda", generator=g, dtype=torch.uint8)  # c·a of c >= 4: above 2^128
    d = torch.arange(N, device="cuda", dtype=torch.int32) % 3 - 1
    code[:, at] = (z[at // G].int() + d).to(torch.uint8)
    a = torch.randint(-4, 5, (M, K), device="cuda", generator=g).bfloat16()
    a[row, at] = big
    w = _weights(code, s, z)
    old = torch.randint(-8, 9, (M, N), device="cuda", generator=g).float()
    for beta in (0.0, 0.5):
        exact = a.double() @ w.t().contiguous() + beta * old.double()
        got = ops.w4_gemm(a, _pack(code), s, z, out_dtype="f32", out=old.clone(), beta=beta).double()
        bound = (K + 3 * (K // G) + 16) * 2.0 ** -23 * (a[row].double().abs() @ w.abs().t().contiguous() + old[row].abs())
        assert bool(((got[row] - exact[row]).abs() <= bound).all())
        same = d == 0
        assert int(same.sum()) > 100 and torch.equal(got[row][same], exact[row][same])  # whole quarters below 2^20
        rest = [r for r in range(M) if r != row]
        assert torch.equal(got[rest], exact[rest])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N", [(9, 400), (60, 32800)])
def test_activations_of_one_sign(M, N, dtype):
    """Codes at or near their zero under activations of one sign: fp16 takes the zero off each code, so its sums are
    off by their bound over |a|·|s|·|c - z|, and a W of zeros gives zeros; bf16 takes it off the group's sums, with the
    bound over |a|·|s|·(c + z) that the header states."""
    ops = _ops()
    K, G = 1152, 64
    g = _gen(M + K)
    a = (torch.randn((M, K), device="cuda", generator=g).clamp(min=0) ** 2).to(TORCH[dtype])
    s = (0.5 + torch.rand((K // G, N), device="cuda", generator=g)).to(TORCH[dtype])
    z = torch.randint(0, 16, (K // G, N), device="cuda", generator=g, dtype=torch.uint8)
    at_zero = z.t().repeat_interleave(G, -1)
    some = torch.rand((N, K), device="cuda", generator=g) < 0.05
    code = torch.where(some, torch.randint(0, 16, (N, K), device="cuda", generator=g, dtype=torch.uint8), at_zero)
    for c in (code, at_zero.contiguous()):
        w = _weights(c, s, z)
        exact = a.double() @ w.t().contiguous()
        got = ops.w4_gemm(a, _pack(c), s, z, out_dtype="f32").double()
        size = _weights(c, s, z, True) if dtype == "bf16" else w.abs()
        acc = (K + 3 * (K // G) + 16) * 2.0 ** -23 * (a.double().abs() @ size.t().contiguous())
        assert bool(((got - exact).abs() <= acc + 2.0 ** -24 * (exact.abs() + acc)).all())


# ---- the layout as the README fills it ----------------------------------------------------------------

@gpu
@pytest.mark.parametrize("N,K,group", [(50, 160, 32), (33, 256, 128), (64, 192, 64)])
def test_readme_quantises_and_multiplies(N, K, group):
    """The README's lines: W comes back within half a step of its group and what the scale's rounding adds, and the
    product is W's."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    block = next(b for b in open(os.path.join(root, "README.md")).read().split("```python\n")[1:] if "w4_gemm(" in b)
    g = _gen(N)
    env = dict(torch=torch, N=N, K=K, group=group, w=torch.randn((N, K), device="cuda", generator=g),
               x=torch.randn((7, K), device="cuda", generator=g).bfloat16())
    exec(block.split("```")[0], env)
    code, scales, zeros = env["code"], env["scales"], env["zeros"]
    w = _weights(code, scales, zeros)
    steps = scales.double().t().repeat_interleave(group, -1)
    # a code is off by half a step; at the upper end, where it ends at 15, by half a step of the zero's rounding and
    # by the 15·2^-8 / (1 - 2^-8) steps that a scale rounded down to bf16 leaves out (1e-3: the fp32 quotients)
    assert bool(((w - env["w"].double()).abs() <= (0.5 + 15 / 255 + 1e-3) * steps).all())
    exact = env["x"].double() @ w.t().contiguous()
    assert bool(((env["y"].double() - exact).abs() <= _bound(env["x"], code, scales, zeros, exact, "bf16")).all())
