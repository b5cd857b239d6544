"""Torch-facing helpers over the C ABI: device memory and streams come from PyTorch, every step
of the computation runs in the library's kernels.  Marshalling only."""
from __future__ import annotations

from typing import Optional, Sequence

import torch

import tiled_bf16_gemm_amd as tbg

_AB_OF = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float8_e4m3fn: "f8e4m3", torch.float8_e5m2: "f8e5m2"}
_TORCH_OF = {"u8": torch.uint8, "u16": torch.int16, "u32": torch.int32, "f16": torch.float16,
             "bf16": torch.bfloat16, "f32": torch.float32}
_X_OF = {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}


def stream_handle(stream: Optional[torch.cuda.Stream] = None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _require(t: torch.Tensor, name: str, device: Optional[torch.device] = None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D row-major view (unit inner stride)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, A on {device}: every operand must be on one device")


# tbg_gemm_workspace_query's answers.  The query reads the sizes, the operand type and layout, the
# leading dimensions and only the operands' addresses modulo 16 (their 16-byte alignment), so
# that is the key; the table is cleared when it grows past a few thousand shapes.
_WS_NEED: dict = {}


def _gemm_workspace_need(M, N, K, ab, a_ptr, lda, b_ptr, ldb, b_layout) -> int:
    key = (M, N, K, ab, a_ptr & 15, lda, b_ptr & 15, ldb, b_layout)
    need = _WS_NEED.get(key)
    if need is None:
        if len(_WS_NEED) > 4096:
            _WS_NEED.clear()
        need = _WS_NEED[key] = tbg.gemm_workspace_query(M, N, K, ab, a_ptr, lda, b_ptr, ldb, b_layout)
    return need


def _require_workspace(ws: Optional[torch.Tensor], device: torch.device):
    if ws is not None and (not ws.is_cuda or ws.device != device or not ws.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous CUDA tensor on {device}")


def gemm(A: torch.Tensor, B: torch.Tensor, b_layout: str = "kn", out_dtype: str = "bf16",
         out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
         stream: Optional[torch.cuda.Stream] = None, alpha: float = 1.0, beta: float = 0.0,
         config: Optional[tbg.GemmConfig] = None) -> torch.Tensor:
    """C = alpha·A·B + beta·C through tbg_gemm (alpha = 1, beta = 0), tbg_gemm_ex, or
    tbg_gemm_configured when `config` (tbg.gemm_config(...)) is given; fp16 and 8-bit float
    operands (float8_e4m3fn, float8_e5m2; B stored "nk" only) go through tbg_gemm_typed.
    A: (M, K) view; B: (K, N) for "kn" or (N, K) for "nk".  Row strides become the leading
    dimensions.  `out` (M, N) may be a strided view; with beta != 0 it must hold the old C."""
    _require(A, "A")
    _require(B, "B", A.device)
    ab = _AB_OF.get(A.dtype)
    if ab is None or B.dtype != A.dtype:
        raise ValueError("A and B must have the same dtype: bfloat16, float16, float8_e4m3fn or float8_e5m2")
    M, K = A.shape
    if b_layout == "kn":
        Kb, N = B.shape
    else:
        N, Kb = B.shape
    if Kb != K:
        raise ValueError(f"inner sizes differ: {K} vs {Kb}")
    if out_dtype not in ("f32", "bf16"):
        raise ValueError(f"out_dtype must be 'f32' or 'bf16' (got {out_dtype!r})")
    if out is None:
        out = torch.empty((M, N), dtype=_TORCH_OF[out_dtype], device=A.device)
    _require(out, "out", A.device)
    # the kernel writes M rows of N elements of out_dtype at out's row stride: out must be exactly that
    if tuple(out.shape) != (M, N) or out.dtype != _TORCH_OF[out_dtype]:
        raise ValueError(f"out must be a ({M}, {N}) {_TORCH_OF[out_dtype]} view (got {tuple(out.shape)} {out.dtype})")
    _require_workspace(workspace, A.device)
    lda, ldb, ldc = A.stride(0), B.stride(0), out.stride(0)
    a_ptr, b_ptr, c_ptr = A.data_ptr(), B.data_ptr(), out.data_ptr()
    need = _gemm_workspace_need(M, N, K, ab, a_ptr, lda, b_ptr, ldb, b_layout)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if need and ws_bytes < need:
        # twice the need: successive calls alternate the halves their repacks land in
        workspace = torch.empty(2 * need, dtype=torch.uint8, device=A.device)
        ws_bytes = 2 * need
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    s = stream_handle(stream)
    if ab != "bf16":
        tbg.gemm_typed(M, N, K, alpha, a_ptr, lda, b_ptr, ldb, b_layout, ab, beta, c_ptr, ldc, out_dtype, config,
                       ws_ptr, ws_bytes, s)
    elif config is not None:
        tbg.gemm_configured(M, N, K, alpha, a_ptr, lda, b_ptr, ldb, b_layout, beta, c_ptr, ldc, out_dtype, config,
                            ws_ptr, ws_bytes, s)
    elif alpha == 1.0 and beta == 0.0:
        tbg.gemm(M, N, K, a_ptr, lda, b_ptr, ldb, b_layout, c_ptr, ldc, out_dtype, ws_ptr, ws_bytes, s)
    else:
        tbg.gemm_ex(M, N, K, alpha, a_ptr, lda, b_ptr, ldb, b_layout, beta, c_ptr, ldc, out_dtype, ws_ptr, ws_bytes, s)
    return out


# ---- ragged groups and microscaled 4-bit data ------------------------------------------------------

# These calls check a tensor's place by its device number (get_device(), -1 on the host).

class _Launch:
    """One call's place: device number `index` current, and what the call allocates on `stream`
    (default: that device's current stream).  Gives the stream's handle."""
    __slots__ = ("handle", "ctx")

    def __init__(self, index: int, stream: Optional[torch.cuda.Stream]):
        if stream is None:
            # (raw calls: building a torch.cuda.Stream object costs 1.8 us, current_device() 0.3)
            self.ctx = None if index == torch._C._cuda_getDevice() else torch.cuda.device(index)
            self.handle = torch._C._cuda_getCurrentRawStream(index)
        else:
            if stream.device.index != index:
                raise ValueError(f"stream is on {stream.device}, the operands on cuda:{index}")
            self.ctx = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream

    def __enter__(self) -> int:
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _require_offsets(offsets: torch.Tensor, index: int) -> int:
    if offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous() or offsets.shape[0] < 1:
        raise ValueError("offsets must be a contiguous 1-D int32 CUDA tensor of groups + 1 values")
    if offsets.get_device() != index:
        raise ValueError(f"offsets is on {offsets.device}, the operands on cuda:{index}")
    return offsets.shape[0] - 1


def _require_rows(t: torch.Tensor, name: str, index: int, dims: int = 2):
    """A row-major matrix (dims 2) or stack of matrices (3) on device `index`; its shape and strides."""
    shape, strides = t.shape, t.stride()
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} is on {t.device}: every operand must be on one CUDA (HIP) device")
    if len(shape) != dims or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError(f"{name} must be a {dims}-D row-major view (unit inner stride)")
    return shape, strides


def _pitch(shape, strides) -> int:
    """Row stride of a matrix, or of each matrix of a stack.  A single row's is never used, and torch may
    call it anything (a token of a long sequence: past the largest leading dimension): its length, rounded
    up to 8 values, stands in for it."""
    return strides[-2] if shape[-2] > 1 else max(-(-shape[-1] // 8) * 8, 1)


def _output(out: Optional[torch.Tensor], shape, out_dtype: str, allowed, index: int, beta: float = 0.0) -> torch.Tensor:
    """The caller's `out`, checked, or a new tensor (which holds no C that beta could scale)."""
    if out_dtype not in allowed:
        raise ValueError(f"out_dtype must be one of {', '.join(allowed)} (got {out_dtype!r})")
    dtype = _TORCH_OF[out_dtype]
    if out is None:
        if beta != 0.0:
            raise ValueError(f"beta={beta} needs out, which holds the old C")
        return torch.empty(*shape, dtype=dtype, device=index)  # (as a tuple, the sizes take 0.36 us more)
    if out.dtype != dtype or tuple(out.shape) != shape or out.get_device() != index:
        raise ValueError(f"out must be a {shape} {dtype} tensor on cuda:{index} (got {tuple(out.shape)} {out.dtype} on "
                         f"{out.device})")
    if out.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError("out must have a unit inner stride")
    return out


def _workspace(need: int, workspace: Optional[torch.Tensor], device: torch.device):
    """(address, bytes) of the caller's workspace where it suffices, else of a new one (returned last,
    to be held until the call is enqueued)."""
    if workspace is None:
        if need == 0:
            return 0, 0, None
    else:
        _require_workspace(workspace, device)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        # twice the need: successive calls alternate the halves their repacks land in
        workspace = torch.empty(2 * need, dtype=torch.uint8, device=device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def gemm_grouped(A: torch.Tensor, B: torch.Tensor, offsets: torch.Tensor, b_layout: str = "kn",
                 out_dtype: str = "bf16", out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None, alpha: float = 1.0, beta: float = 0.0) -> torch.Tensor:
    """C[r] = alpha·A[r]·B[e] + beta·C[r] for the rows r of every group e (offsets[e] <= r <
    offsets[e+1]) through tbg_gemm_grouped.  A: (M, K) bf16 or fp16; B: (groups, K, N) for "kn" or
    (groups, N, K) for "nk"; offsets: (groups + 1,) int32 on the device.  out_dtype: "f32" or A's
    type.  Rows of no group keep what `out` holds (without `out`: undefined); beta != 0 needs `out`.
    Gradients, for dC of C's shape: of the rows gemm_grouped(dC, B, offsets, the other layout), of B
    gemm_grouped_wgrad(A, dC, offsets) for "kn" and gemm_grouped_wgrad(dC, A, offsets) for "nk"."""
    index = A.get_device()
    (M, K), st_a = _require_rows(A, "A", index)
    shape_b, st_b = _require_rows(B, "B", index, 3)
    groups = _require_offsets(offsets, index)
    ab = _AB_OF.get(A.dtype)
    if ab not in ("bf16", "f16") or B.dtype != A.dtype:
        raise ValueError("A and B must have the same dtype: bfloat16 or float16")
    if b_layout == "nk":
        matrices, N, Kb = shape_b
    elif b_layout == "kn":
        matrices, Kb, N = shape_b
    else:
        raise ValueError(f"b_layout must be 'kn' or 'nk' (got {b_layout!r})")
    if Kb != K:
        raise ValueError(f"inner sizes differ: {K} vs {Kb}")
    if matrices != groups:
        raise ValueError(f"B holds {matrices} matrices, offsets {groups} groups")
    with _Launch(index, stream) as handle:
        out = _output(out, (M, N), out_dtype, ("f32", ab), index, beta)
        a, b = A.data_ptr(), B.data_ptr()
        lda, ldb, sb = _pitch((M, K), st_a), _pitch(shape_b, st_b), st_b[0]
        # whole 16-byte rows everywhere need no repack; the query knows the exact rule
        need = 0 if (lda | ldb | sb | K) % 8 == 0 and (a | b) % 16 == 0 else \
            tbg.gemm_grouped_workspace_query(groups, M, N, K, ab, a, lda, b, ldb, sb, b_layout)
        ws_ptr, ws_bytes, held = _workspace(need, workspace, A.device)
        tbg.gemm_grouped(groups, M, N, K, offsets.data_ptr(), alpha, a, lda, b, ldb, sb, b_layout, ab, beta,
                         out.data_ptr(), _pitch((M, N), out.stride()), out_dtype, ws_ptr, ws_bytes, handle)
    return out


def gemm_grouped_wgrad(X: torch.Tensor, Y: torch.Tensor, offsets: torch.Tensor, out_dtype: str = "f32",
                       out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None, alpha: float = 1.0,
                       beta: float = 0.0) -> torch.Tensor:
    """C[e] = alpha·X[rows of e]ᵀ·Y[rows of e] + beta·C[e] through tbg_gemm_grouped_wgrad.  X: (M, P),
    Y: (M, Q), bf16 or fp16; out: (groups, P, Q) of type "f32" or X's, needed when beta != 0.  An empty
    group's C is beta·C (zeros when beta == 0)."""
    index = X.get_device()
    (M, P), st_x = _require_rows(X, "X", index)
    (My, Q), st_y = _require_rows(Y, "Y", index)
    groups = _require_offsets(offsets, index)
    ab = _AB_OF.get(X.dtype)
    if ab not in ("bf16", "f16") or Y.dtype != X.dtype:
        raise ValueError("X and Y must have the same dtype: bfloat16 or float16")
    if My != M:
        raise ValueError(f"X has {M} rows, Y {My}")
    with _Launch(index, stream) as handle:
        out = _output(out, (groups, P, Q), out_dtype, ("f32", ab), index, beta)
        x, y, st_c = X.data_ptr(), Y.data_ptr(), out.stride()
        ldx, ldy = _pitch((M, P), st_x), _pitch((M, Q), st_y)
        need = 0 if (ldx | ldy) % 8 == 0 and (x | y) % 16 == 0 else \
            tbg.gemm_grouped_wgrad_workspace_query(groups, M, P, Q, ab, x, ldx, y, ldy)
        ws_ptr, ws_bytes, held = _workspace(need, workspace, X.device)
        tbg.gemm_grouped_wgrad(groups, M, P, Q, offsets.data_ptr(), alpha, x, ldx, y, ldy, ab, beta, out.data_ptr(),
                               _pitch((P, Q), st_c[1:]), st_c[0], out_dtype, ws_ptr, ws_bytes, handle)
    return out


def _require_mx4(codes: torch.Tensor, scales: torch.Tensor, name: str, index: int, dims=(2, 3)):
    """Codes and scales that belong together, on device `index`: the codes' shape and both pitches in
    bytes (a single row's pitch is its length rounded up to 16, that of rows without a value 0)."""
    shape, blocks, st, st_s = codes.shape, scales.shape, codes.stride(), scales.stride()
    if codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8:
        raise ValueError(f"{name}'s codes and scales must be uint8 tensors")
    if index < 0 or codes.get_device() != index or scales.get_device() != index:
        raise ValueError(f"{name} is on {codes.device} and {scales.device}: every operand must be on one CUDA (HIP) "
                         "device")
    n = len(shape)
    if n not in dims or len(blocks) != n:
        raise ValueError(f"{name}'s codes and scales must have {' or '.join(map(str, dims))} dimensions")
    rows, half = shape[-2:]
    nb = blocks[-1]
    if half != 16 * nb or blocks[-2] != rows or blocks[0] != shape[0]:
        raise ValueError(f"{name}: codes {tuple(shape)} and scales {tuple(blocks)} do not belong together (16 bytes of "
                         "codes and one scale per 32 values)")
    if (st[-1] != 1 and half > 1) or (st_s[-1] != 1 and nb > 1):
        raise ValueError(f"{name}'s codes and scales must have a unit inner stride")
    if rows > 1 and half > 0:
        return shape, st[-2], st_s[-2]
    return shape, half, -(-nb // 16) * 16


def _flat_rows(t: torch.Tensor, name: str) -> torch.Tensor:
    """A matrix, or the 2-D view of a stack of matrices whose rows lie at one pitch."""
    if t.dim() == 2:
        return t
    n, rows, cols = t.shape
    if rows == 1:
        return t[:, 0]
    if n > 1 and rows > 0 and t.stride(0) != rows * t.stride(1):
        raise ValueError(f"{name}: the matrices of a stack must follow one another at the rows' pitch")
    return t.as_strided((n * rows, cols), (t.stride(1), t.stride(2)))


def _mx4_rows(codes: torch.Tensor, scales: torch.Tensor, index: int):
    """Rows, codes and scales of a matrix or a stack as one matrix: (rows, codes address, pitch, scales
    address, pitch)."""
    codes, scales = _flat_rows(codes, "codes"), _flat_rows(scales, "scales")
    shape, ld_c, ld_s = _require_mx4(codes, scales, "codes", index, (2,))
    return shape[0], codes.data_ptr(), ld_c, scales.data_ptr(), ld_s


def mx4_quantize(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None):
    """Rows of x, (rows, cols) or a stack (n, rows, cols) of fp32, bf16 or fp16, as microscaled 4-bit
    data through tbg_mx4_quantize.  Returns (codes, scales), uint8: two codes per byte, one scale per
    32 values, cols rounded up to whole blocks (zeros).  The scales' rows are 16-byte pitched."""
    index, x_dtype = x.get_device(), _X_OF.get(x.dtype)
    if index < 0 or x.dim() not in (2, 3) or x_dtype is None:
        raise ValueError("x must be a 2-D or 3-D float32, bfloat16 or float16 CUDA tensor")
    x2 = _flat_rows(x, "x")
    (rows, cols), st = x2.shape, x2.stride()
    if st[1] != 1 and cols > 1:
        raise ValueError("x must have a unit inner stride")
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales must be given together")
    blocks = -(-cols // 32)
    with _Launch(index, stream) as handle:
        if codes is None:
            ld_c, ld_s = 16 * blocks, -(-blocks // 16) * 16
            codes = torch.empty((rows, ld_c), dtype=torch.uint8, device=index)
            scales = torch.empty_strided((rows, blocks), (ld_s, 1), dtype=torch.uint8, device=index)
            c, s = codes.data_ptr(), scales.data_ptr()
            if x2 is not x:
                n, per = x.shape[0], x.shape[1]
                codes = codes.view(n, per, ld_c)
                scales = scales.as_strided((n, per, blocks), (per * ld_s, ld_s, 1))
        else:
            if tuple(codes.shape) != (*x.shape[:-1], 16 * blocks):
                raise ValueError(f"codes must be {(*x.shape[:-1], 16 * blocks)} (got {tuple(codes.shape)})")
            _, c, ld_c, s, ld_s = _mx4_rows(codes, scales, index)
        tbg.mx4_quantize(rows, cols, x2.data_ptr(), _pitch((rows, cols), st), x_dtype, c, ld_c, s, ld_s, handle)
    return codes, scales


def mx4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: Optional[int] = None, out_dtype: str = "bf16",
                   out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values of mx4_quantize's codes and scales through tbg_mx4_dequantize: the first `cols`
    columns (default: all), of type "f32", "bf16" or "f16"."""
    index = codes.get_device()
    shape, ld_c, ld_s = _require_mx4(codes, scales, "codes", index)
    *lead, half = shape
    cols = 2 * half if cols is None else int(cols)
    if not (2 * half - 32 < cols <= 2 * half):
        raise ValueError(f"cols must end in the last block of 32: {max(0, 2 * half - 31)}..{2 * half} (got {cols})")
    with _Launch(index, stream) as handle:
        out = _output(out, (*lead, cols), out_dtype, ("f32", "bf16", "f16"), index)
        o2, rows, c, s = out, shape[0], codes.data_ptr(), scales.data_ptr()
        if len(shape) == 3:
            o2 = _flat_rows(out, "out")
            rows, c, ld_c, s, ld_s = _mx4_rows(codes, scales, index)
        tbg.mx4_dequantize(rows, cols, c, ld_c, s, ld_s, o2.data_ptr(), _pitch(o2.shape, o2.stride()), out_dtype,
                           handle)
    return out


def mx4_gemm(A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor, out_dtype: str = "bf16",
             out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None, alpha: float = 1.0,
             beta: float = 0.0) -> torch.Tensor:
    """C = alpha·A·Bᵀ + beta·C for microscaled 4-bit A (M, K/2 codes) and B (N, K/2 codes), each with
    its scales (rows, K/32), through tbg_mx4_gemm.  Codes and scales 16-byte aligned and pitched, as
    mx4_quantize makes them; beta != 0 needs `out`."""
    index = A.get_device()
    (M, half), lda, ld_as = _require_mx4(A, a_scales, "A", index, (2,))
    (N, half_b), ldb, ld_bs = _require_mx4(B, b_scales, "B", index, (2,))
    if half != half_b:
        raise ValueError(f"inner sizes differ: {2 * half} vs {2 * half_b}")
    with _Launch(index, stream) as handle:
        out = _output(out, (M, N), out_dtype, ("f32", "bf16"), index, beta)
        tbg.mx4_gemm(M, N, 2 * half, alpha, A.data_ptr(), lda, a_scales.data_ptr(), ld_as, B.data_ptr(), ldb,
                     b_scales.data_ptr(), ld_bs, beta, out.data_ptr(), _pitch((M, N), out.stride()), out_dtype, handle)
    return out


def mx4_gemm_grouped(A: torch.Tensor, a_scales: torch.Tensor, B: torch.Tensor, b_scales: torch.Tensor,
                     offsets: torch.Tensor, out_dtype: str = "bf16", out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None, alpha: float = 1.0, beta: float = 0.0) -> torch.Tensor:
    """mx4_gemm for the rows of every group (offsets as gemm_grouped) with its own B, (groups, N, K/2
    codes), through tbg_mx4_gemm_grouped.  Rows of no group keep what `out` holds (without `out`:
    undefined); beta != 0 needs `out`."""
    index = A.get_device()
    (M, half), lda, ld_as = _require_mx4(A, a_scales, "A", index, (2,))
    (matrices, N, half_b), ldb, ld_bs = _require_mx4(B, b_scales, "B", index, (3,))
    groups = _require_offsets(offsets, index)
    if half != half_b:
        raise ValueError(f"inner sizes differ: {2 * half} vs {2 * half_b}")
    if matrices != groups:
        raise ValueError(f"B holds {matrices} matrices, offsets {groups} groups")
    with _Launch(index, stream) as handle:
        out = _output(out, (M, N), out_dtype, ("f32", "bf16"), index, beta)
        tbg.mx4_gemm_grouped(groups, M, N, 2 * half, offsets.data_ptr(), alpha, A.data_ptr(), lda, a_scales.data_ptr(),
                             ld_as, B.data_ptr(), ldb, B.stride(0), b_scales.data_ptr(), ld_bs, b_scales.stride(0),
                             beta, out.data_ptr(), _pitch((M, N), out.stride()), out_dtype, handle)
    return out


# ---- tokens by expert ------------------------------------------------------------------------------

_ELEMENT_OF = {1: "u8", 2: "u16", 4: "u32"}


def _require_ints(t: torch.Tensor, name: str, index: int):
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} is on {t.device}: every operand must be on one CUDA (HIP) device")


def _require_place(place: torch.Tensor, weights: Optional[torch.Tensor], index: int):
    """(tokens, top_k) of place, and the weights that belong to it."""
    _require_ints(place, "place", index)
    shape = place.shape
    if len(shape) != 2:
        raise ValueError("place must be (tokens, top_k)")
    if weights is not None and (weights.dtype != torch.float32 or weights.shape != shape or
                                weights.get_device() != index or not weights.is_contiguous()):
        raise ValueError(f"weights must be a contiguous float32 tensor of place's shape {tuple(shape)} and device")
    return shape


def _pitch_of(out: torch.Tensor, rows: int, cols: int) -> int:
    """Row stride of a checked matrix; a single row's is its length (_pitch)."""
    return out.stride(0) if rows > 1 else cols or 1


def expert_sort(experts: torch.Tensor, groups: int, workspace: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None):
    """A router's choices, int32 (tokens, top_k) or (slots,), sorted by expert through tbg_expert_sort.
    Returns int32 (offsets, source, place): offsets (groups + 1,) of the ragged products, source (slots,)
    with the slot token·top_k + choice of every row (-1 behind the last group), place of experts' shape
    with the row of every slot (-1: an expert outside 0..groups-1, a padded or dropped slot)."""
    index = experts.get_device()
    _require_ints(experts, "experts", index)
    slots = experts.numel()
    with _Launch(index, stream) as handle:
        offsets = experts.new_empty(groups + 1)
        place = torch.empty_like(experts)
        source = torch.empty_like(experts) if experts.dim() == 1 else experts.new_empty(slots)
        ws_ptr = ws_bytes = 0
        if slots > 512:  # fewer need none
            need = tbg.expert_sort_workspace_query(slots, groups)
            ws_ptr, ws_bytes, held = _workspace(need, workspace, experts.device)
        tbg.expert_sort(slots, groups, experts.data_ptr(), offsets.data_ptr(), source.data_ptr(), place.data_ptr(), ws_ptr,
                        ws_bytes, handle)
    return offsets, source, place


def expert_dispatch(X: torch.Tensor, place: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[place[t, j]] = X[t] through tbg_expert_dispatch: the rows of the groups.  X: (tokens, cols) of
    1-, 2- or 4-byte elements (mx4_quantize's codes and scales among them); place as expert_sort gives it.
    Rows that no slot holds keep what `out` holds (without `out`, which has a row for every slot:
    undefined).  The gradient of X is expert_combine(dout, place)."""
    index = X.get_device()
    (tokens, cols), st = _require_rows(X, "X", index)
    placed, top_k = _require_place(place, None, index)
    size = X.element_size()
    if placed != tokens:
        raise ValueError(f"X has {tokens} tokens, place {placed}")
    if size not in _ELEMENT_OF:
        raise ValueError(f"X must have elements of 1, 2 or 4 bytes (got {X.dtype})")
    with _Launch(index, stream) as handle:
        if out is None:
            rows, ld_out = tokens * top_k, cols
            out = X.new_empty(rows, cols)
        else:
            (rows, out_cols), st_o = _require_rows(out, "out", index)
            if out.dtype != X.dtype or out_cols != cols:
                raise ValueError(f"out must be (rows, {cols}) {X.dtype} (got {tuple(out.shape)} {out.dtype})")
            ld_out = st_o[0] if rows > 1 else cols
        tbg.expert_dispatch(tokens, top_k, rows, cols, _ELEMENT_OF[size], X.data_ptr(), st[0] if tokens > 1 else cols,
                            place.data_ptr(), out.data_ptr(), ld_out, handle)
    return out


def expert_combine(Y: torch.Tensor, place: torch.Tensor, weights: Optional[torch.Tensor] = None,
                   out_dtype: Optional[str] = None, out: Optional[torch.Tensor] = None,
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out[t] = sum over j of weights[t, j]·Y[place[t, j]] through tbg_expert_combine.  Y: (rows, cols) fp32,
    bf16 or fp16; place as expert_sort gives it (a slot without a row adds nothing); weights: float32 of
    place's shape, or None for ones.  out_dtype: "f32" or Y's type (default).  Gradients:
    expert_combine_grad."""
    index = Y.get_device()
    (rows, cols), st = _require_rows(Y, "Y", index)
    tokens, top_k = _require_place(place, weights, index)
    y_dtype = _X_OF.get(Y.dtype)
    if y_dtype is None:
        raise ValueError("Y must be float32, bfloat16 or float16")
    out_dtype = out_dtype or y_dtype
    with _Launch(index, stream) as handle:
        out = _output(out, (tokens, cols), out_dtype, ("f32", y_dtype), index)
        tbg.expert_combine(tokens, top_k, rows, cols, Y.data_ptr(), st[0] if rows > 1 else cols, y_dtype, place.data_ptr(),
                           weights.data_ptr() if weights is not None else 0, out.data_ptr(),
                           _pitch_of(out, tokens, cols), out_dtype, handle)
    return out


def expert_combine_grad(dout: torch.Tensor, Y: torch.Tensor, place: torch.Tensor, weights: Optional[torch.Tensor] = None,
                        dy: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None):
    """(dY, dweights) of expert_combine(Y, place, weights) for the gradient dout, (tokens, cols) of float32 or
    Y's type, through tbg_expert_combine_grad: dY[place[t, j]] = weights[t, j]·dout[t] in Y's type (rows that no
    slot holds keep what `dy` holds, without `dy`: undefined), dweights[t, j] = Y[place[t, j]]·dout[t] in
    float32 (0 for a slot without a row)."""
    index = Y.get_device()
    (rows, cols), st = _require_rows(Y, "Y", index)
    shape_d, st_d = _require_rows(dout, "dout", index)
    tokens, top_k = _require_place(place, weights, index)
    y_dtype, d_dtype = _X_OF.get(Y.dtype), _X_OF.get(dout.dtype)
    if y_dtype is None or d_dtype not in ("f32", y_dtype):
        raise ValueError("Y must be float32, bfloat16 or float16, dout float32 or Y's type")
    if tuple(shape_d) != (tokens, cols):
        raise ValueError(f"dout must be {(tokens, cols)} (got {tuple(shape_d)})")
    with _Launch(index, stream) as handle:
        dy = _output(dy, (rows, cols), y_dtype, (y_dtype,), index)
        dweights = torch.empty(tokens, top_k, dtype=torch.float32, device=index)
        tbg.expert_combine_grad(tokens, top_k, rows, cols, dout.data_ptr(), st_d[0] if tokens > 1 else cols, d_dtype,
                                Y.data_ptr(), st[0] if rows > 1 else cols, y_dtype, place.data_ptr(),
                                weights.data_ptr() if weights is not None else 0, dy.data_ptr(),
                                _pitch_of(dy, rows, cols), dweights.data_ptr(), handle)
    return dy, dweights


# ---- weights in 4-bit codes ------------------------------------------------------------------------

def _require_w4(codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor], a_dtype, index: int, dims: int):
    """A matrix (dims 2) or stack of matrices (3) in 4-bit codes: its shape (…, N, K), the group, and the
    pitches and strides of codes, scales and zeros."""
    shape, st = _require_rows(codes, "codes", index, dims)
    shape_s, st_s = _require_rows(scales, "scales", index, dims)
    if codes.dtype is not torch.uint8 or scales.dtype is not a_dtype:
        raise ValueError(f"codes must be uint8 and scales of A's type {a_dtype} (got {codes.dtype}, {scales.dtype})")
    N, K = shape[-2], 2 * shape[-1]
    parts = shape_s[-2]
    if shape_s[-1] != N or shape_s[0] != (shape[0] if dims == 3 else parts):
        raise ValueError(f"scales {tuple(shape_s)} do not belong to codes {tuple(shape)}")
    if (parts == 0) != (K == 0) or (parts and (K % parts or K // parts not in (32, 64, 128))):
        raise ValueError(f"K={K} over {parts} rows of scales: groups must be of 32, 64 or 128")
    if zeros is None:
        z, ld_z, stride_z = 0, 0, 0
    else:
        shape_z, st_z = _require_rows(zeros, "zeros", index, dims)
        if zeros.dtype is not torch.uint8 or shape_z != shape_s:
            raise ValueError(f"zeros must be uint8 of scales' shape {tuple(shape_s)}")
        z, ld_z, stride_z = zeros.data_ptr(), st_z[-2] if parts > 1 else max(N, 1), st_z[0]
    return (N, K, K // parts if parts else 32, codes.data_ptr(), st[-2] if N > 1 and K > 0 else max(-(-K // 32), 1) * 16, st[0],
            scales.data_ptr(), st_s[-2] if parts > 1 else max(N, 1), st_s[0], z, ld_z, stride_z)


def w4_gemm(A: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None,
            out_dtype: str = "bf16", out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
            alpha: float = 1.0, beta: float = 0.0) -> torch.Tensor:
    """C = alpha·A·Wᵀ + beta·C for weights in 4-bit codes through tbg_w4_gemm.  A: (M, K) bf16 or fp16; codes:
    (N, K/2) uint8, the lower nibble first, 16-byte aligned and pitched; scales: (K/group, N) of A's type and
    zeros: (K/group, N) uint8 or None (every zero is 8), group 32, 64 or 128:
    W[n, k] = scales[k//group, n]·(code[n, k] - zeros[k//group, n]).  out_dtype: "f32" or A's type; beta != 0
    needs `out`.  For bf16 the fp32 sums' error goes with |a|·|scale|·(code + zero) (tbg_w4_gemm)."""
    index = A.get_device()
    (M, Ka), st_a = _require_rows(A, "A", index)
    ab = _AB_OF.get(A.dtype)
    if ab not in ("bf16", "f16"):
        raise ValueError("A must be bfloat16 or float16")
    N, K, group, c, ldb, _, s, ld_s, _, z, ld_z, _ = _require_w4(codes, scales, zeros, A.dtype, index, 2)
    if Ka != K:
        raise ValueError(f"inner sizes differ: {Ka} vs {K}")
    with _Launch(index, stream) as handle:
        out = _output(out, (M, N), out_dtype, ("f32", ab), index, beta)
        tbg.w4_gemm(M, N, K, group, alpha, A.data_ptr(), st_a[0] if M > 1 else K or 1, ab, c, ldb, s, ld_s, z, ld_z, beta,
                    out.data_ptr(), _pitch_of(out, M, N), out_dtype, handle)
    return out


def w4_gemm_grouped(A: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, offsets: torch.Tensor,
                    zeros: Optional[torch.Tensor] = None, source: Optional[torch.Tensor] = None, top_k: int = 1,
                    out_dtype: str = "bf16", out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None, alpha: float = 1.0, beta: float = 0.0) -> torch.Tensor:
    """w4_gemm for the rows of every group (offsets as gemm_grouped) with its own W, codes (groups, N, K/2),
    scales and zeros (groups, K/group, N), through tbg_w4_gemm_grouped.  With `source` (expert_sort's, one slot
    a row) row r reads A[source[r] // top_k]: the experts' rows of A's tokens without a copy.  Rows of no group
    keep what `out` holds (without `out`: undefined); beta != 0 needs `out`."""
    index = A.get_device()
    (a_rows, Ka), st_a = _require_rows(A, "A", index)
    ab = _AB_OF.get(A.dtype)
    if ab not in ("bf16", "f16"):
        raise ValueError("A must be bfloat16 or float16")
    groups = _require_offsets(offsets, index)
    N, K, group, c, ldb, sb, s, ld_s, ss, z, ld_z, sz = _require_w4(codes, scales, zeros, A.dtype, index, 3)
    if Ka != K:
        raise ValueError(f"inner sizes differ: {Ka} vs {K}")
    if codes.shape[0] != groups:
        raise ValueError(f"codes hold {codes.shape[0]} matrices, offsets {groups} groups")
    M, src = a_rows, 0
    if source is not None:
        _require_ints(source, "source", index)
        if source.dim() != 1:
            raise ValueError("source must be (rows,)")
        M, src = source.shape[0], source.data_ptr()
    with _Launch(index, stream) as handle:
        out = _output(out, (M, N), out_dtype, ("f32", ab), index, beta)
        tbg.w4_gemm_grouped(groups, M, N, K, group, offsets.data_ptr(), src, a_rows, top_k, alpha, A.data_ptr(),
                            st_a[0] if a_rows > 1 else K or 1, ab, c, ldb, sb, s, ld_s, ss, z, ld_z, sz, beta,
                            out.data_ptr(), _pitch_of(out, M, N), out_dtype, handle)
    return out


def encode(t: torch.Tensor, dtype: str, dims: Sequence[int], strides_bytes: Sequence[int], box: Sequence[int],
           estr: Sequence[int], swizzle: str = "none", oob: str = "zero", l2: str = "none") -> tbg.TensorDesc:
    """Descriptor for the tensor whose element (0, ..., 0) is t's first element."""
    return tbg.encode_tiled(dtype, len(dims), t.data_ptr(), dims, list(strides_bytes), box, estr, swizzle, l2, oob)


def tiled_copy(desc: tbg.TensorDesc, coords: Sequence[int], out: Optional[torch.Tensor] = None,
               device="cuda", stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    nbytes = tbg.box_bytes(desc)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=device)
    tbg.tiled_copy(desc, coords, out.data_ptr(), stream_handle(stream))
    return out


def tiled_copy_many(desc: tbg.TensorDesc, coords: torch.Tensor, out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """coords: (n, rank) int32 CUDA tensor.  Returns n images of box_bytes each (uint8, flat)."""
    if coords.dtype != torch.int32 or not coords.is_cuda or not coords.is_contiguous():
        raise ValueError("coords must be a contiguous int32 CUDA tensor")
    n = coords.shape[0]
    nbytes = tbg.box_bytes(desc)
    if out is None:
        out = torch.empty(n * nbytes, dtype=torch.uint8, device=coords.device)
    tbg.tiled_copy_many(desc, coords.data_ptr(), n, out.data_ptr(), stream_handle(stream))
    return out


def tiled_store(desc: tbg.TensorDesc, coords: Sequence[int], image: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> None:
    """Store one box image (a CUDA tensor of box_bytes bytes) into the descriptor's tensor."""
    if not image.is_cuda or image.numel() * image.element_size() < tbg.box_bytes(desc):
        raise ValueError("image must be a CUDA tensor of at least box_bytes bytes")
    tbg.tiled_store(desc, coords, image.data_ptr(), stream_handle(stream))


def tiled_store_many(desc: tbg.TensorDesc, coords: torch.Tensor, images: torch.Tensor,
                     stream: Optional[torch.cuda.Stream] = None) -> None:
    """coords: (n, rank) int32 CUDA tensor; images: n images of box_bytes each, back to back."""
    if coords.dtype != torch.int32 or not coords.is_cuda or not coords.is_contiguous():
        raise ValueError("coords must be a contiguous int32 CUDA tensor")
    n = coords.shape[0]
    if images.numel() * images.element_size() < n * tbg.box_bytes(desc):
        raise ValueError("images holds fewer than n box images")
    tbg.tiled_store_many(desc, coords.data_ptr(), n, images.data_ptr(), stream_handle(stream))


def conv2d(x: torch.Tensor, w: torch.Tensor, pad=(0, 0, 0, 0), stride=(1, 1), dil=(1, 1), out_dtype: str = "bf16",
           out: Optional[torch.Tensor] = None, alpha: float = 1.0, beta: float = 0.0,
           workspace: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None,
           config: Optional[tbg.GemmConfig] = None) -> torch.Tensor:
    """Y = alpha·conv2d(x, w) + beta·Y through tbg_conv2d_fwd.  x: (N, H, W, C) bf16 contiguous
    (NHWC); w: (K, R, S, C) bf16 contiguous (KRSC); pad = (top, left, bottom, right); stride and
    dil = (h, w).  Returns / fills out: (N·OH·OW, K) rows, row stride = ldy."""
    for t, name in ((x, "x"), (w, "w")):
        if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 4-D bfloat16 CUDA tensor")
    n, h, wd, c = x.shape
    k, r, s, c2 = w.shape
    if c2 != c:
        raise ValueError(f"channel counts differ: {c} vs {c2}")
    shp = tbg.conv2d_shape(n, h, wd, c, k, r, s, pad, stride, dil)
    oh, ow = tbg.conv2d_out_dims(shp)
    if out is None:
        out = torch.empty((n * oh * ow, k), dtype=_TORCH_OF[out_dtype], device=x.device)
    if out.dim() != 2 or out.stride(1) != 1 or out.shape[0] != n * oh * ow or out.shape[1] != k:
        raise ValueError("out must be a (N·OH·OW, K) row-major view")
    if w.device != x.device or out.device != x.device:
        raise ValueError("x, w and out must be on one device")
    if out.dtype != _TORCH_OF[out_dtype]:
        raise ValueError(f"out must hold {_TORCH_OF[out_dtype]} for out_dtype {out_dtype!r} (got {out.dtype})")
    _require_workspace(workspace, x.device)
    need = tbg.conv2d_workspace_query(shp, x.data_ptr(), w.data_ptr())
    if need and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(2 * need, dtype=torch.uint8, device=x.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else 0
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    tbg.conv2d_fwd(shp, alpha, x.data_ptr(), w.data_ptr(), beta, out.data_ptr(), out.stride(0), out_dtype, config,
                   ws_ptr, ws_bytes, stream_handle(stream))
    return out


def encode_im2col(t: torch.Tensor, dtype: str, pad=(0, 0, 0, 0), stride=(1, 1), dil=(1, 1), filt=(1, 1),
                  channels: int = 64, pixels: int = 64, swizzle: str = "none", oob: str = "zero") -> tbg.TensorDesc:
    """im2col descriptor of a contiguous NHWC tensor t; pad = (top, left, bottom, right), stride,
    dil and filt = (h, w)."""
    n, h, w, c = t.shape
    es = t.element_size()
    return tbg.encode_im2col(dtype, t.data_ptr(), [c, w, h, n], [c * es, c * es * w, c * es * w * h],
                             [pad[1], pad[0]], [pad[3], pad[2]], [stride[1], stride[0]], [dil[1], dil[0]],
                             [filt[1], filt[0]], channels, pixels, swizzle, "none", oob)


def im2col_copy(desc: tbg.TensorDesc, coords, out: Optional[torch.Tensor] = None, device="cuda",
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    nbytes = tbg.box_bytes(desc)
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=device)
    tbg.im2col_copy(desc, coords, out.data_ptr(), stream_handle(stream))
    return out


def im2col_copy_many(desc: tbg.TensorDesc, coords: torch.Tensor, out: Optional[torch.Tensor] = None,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """coords: (n, 4) int32 CUDA tensor of {c0, m0, s, r}.  Returns n images back to back."""
    if coords.dtype != torch.int32 or not coords.is_cuda or not coords.is_contiguous() or coords.shape[1] != 4:
        raise ValueError("coords must be a contiguous (n, 4) int32 CUDA tensor")
    n = coords.shape[0]
    nbytes = tbg.box_bytes(desc)
    if out is None:
        out = torch.empty(n * nbytes, dtype=torch.uint8, device=coords.device)
    tbg.im2col_copy_many(desc, coords.data_ptr(), n, out.data_ptr(), stream_handle(stream))
    return out
