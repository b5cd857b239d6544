"""Measured cases of the products that serve and train expert layers, and of the 4-bit formats.

Five operators, each with its plain form in elementary torch operations and the call a user's
program makes of this package:

  quantize   x -> microscaled 4-bit values (E2M1 codes, one E8M0 scale per 32) and back to values
  product    C = A·Bᵀ of two microscaled 4-bit matrices
  grouped    C[rows of group e] = A[rows of group e]·B_e, 16-bit operands, ragged groups
  wgrad      C_e = X[rows of group e]ᵀ·Y[rows of group e], the weight gradient of `grouped`
  experts    `grouped` over microscaled 4-bit operands, B_e stored N×K

A case is a dict of plain values; prepare() draws its inputs from the seed alone, run() makes one
pass, exact() gives the definition's value in 64 bits, work() the bytes and operations that a pass
cannot do without.  `own` is False for the plain forms and True for the package's kernels.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases --------------------------------------------------------------------------------------

def listed():
    return [
        # a few rows of an odd width, as a cache or a router holds them: launch latency counts
        dict(name="quantize_7x2049_f16", op="quantize", rows=7, cols=2049, dtype="f16"),
        # one layer's activations of a long prefill
        dict(name="quantize_16384x4096_bf16", op="quantize", rows=16384, cols=4096, dtype="bf16"),
        # one token through a 4-bit weight
        dict(name="product_1x14336x4096", op="product", M=1, N=14336, K=4096, out="bf16"),
        # sizes that overhang every tile, fp32 out
        dict(name="product_3001x2049x800", op="product", M=3001, N=2049, K=800, out="f32"),
        # the large square product
        dict(name="product_8192", op="product", M=8192, N=8192, K=8192, out="bf16"),
        # decoding: 8 tokens, 8 experts each, of 64
        dict(name="grouped_decode_64e", op="grouped", groups=64, active=40, rows=64, tail=0, N=2048, K=4096,
             dtype="bf16", layout="nk", out="bf16"),
        # the forward product of a training step
        dict(name="grouped_8e_16384x14336x4096", op="grouped", groups=8, active=8, rows=16384, tail=0, N=14336, K=4096,
             dtype="bf16", layout="nk", out="bf16"),
        # the gradient of the rows (the weights read the other way), odd inner size, a padded batch
        dict(name="grouped_rows_32e_f16", op="grouped", groups=32, active=31, rows=8001, tail=191, N=2000, K=1001,
             dtype="f16", layout="kn", out="f16"),
        # the weight gradient of many small experts, some of them without a row
        dict(name="wgrad_64e_777x256x200_f16", op="wgrad", groups=64, active=49, rows=777, tail=23, P=256, Q=200,
             dtype="f16", out="f32"),
        # the weight gradient of a training step
        dict(name="wgrad_8e_16384x4096x2048", op="wgrad", groups=8, active=8, rows=16384, tail=0, P=4096, Q=2048,
             dtype="bf16", out="f32"),
        # decoding through 4-bit experts
        dict(name="experts_decode_64e", op="experts", groups=64, active=40, rows=64, tail=0, N=4096, K=2048,
             out="bf16"),
        # a prefill through 4-bit experts, ragged
        dict(name="experts_32e_16000x4096x2048", op="experts", groups=32, active=32, rows=16000, tail=384, N=4096,
             K=2048, out="bf16"),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "grouped", "wgrad", "experts"])
    if op == "quantize":
        rows, cols = _spread(rng, 1, 16384), _spread(rng, 32, 16384)
        while rows * cols > 16384 * 4096:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["bf16", "f16", "f32"]))
    if op == "product":
        return dict(op=op, M=_spread(rng, 1, 8192), N=_spread(rng, 16, 8192), K=BLOCK * _spread(rng, 1, 256),
                    out=rng.choice(["bf16", "f32"]))
    groups = _spread(rng, 1, 128)
    rows = _spread(rng, 1, 16384)
    active = min(rows, rng.randint(max(1, groups // 2), groups))
    tail = rng.choice([0, 0, rng.randint(1, 64)])
    big, small = _spread(rng, 16, 4096), _spread(rng, 16, 2048)
    if rng.random() < 0.5:
        big, small = small, big
    if op == "experts":
        return dict(op=op, groups=groups, active=active, rows=rows, tail=tail, N=big,
                    K=max(BLOCK, small // BLOCK * BLOCK), out=rng.choice(["bf16", "f32"]))
    dtype = rng.choice(["bf16", "f16"])
    if op == "wgrad":
        return dict(op=op, groups=groups, active=active, rows=rows, tail=tail, P=big, Q=small, dtype=dtype,
                    out=rng.choice(["f32", dtype]))
    return dict(op=op, groups=groups, active=active, rows=rows, tail=tail, N=big, K=small, dtype=dtype,
                layout=rng.choice(["nk", "kn"]), out=rng.choice(["f32", dtype]))


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        packed = case["rows"] * (-(-case["cols"] // BLOCK)) * (BLOCK // 2 + 1)
        return {"bytes": 2 * n * SIZE[case["dtype"]] + 2 * packed, "flops": 4 * n}
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * 17 // 32 + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    rows, act = case["rows"], case["active"]
    if op == "wgrad":
        P, Q = case["P"], case["Q"]
        return {"bytes": rows * (P + Q) * 2 + case["groups"] * P * Q * SIZE[case["out"]], "flops": 2 * rows * P * Q}
    N, K = case["N"], case["K"]
    moved = (rows + act * N) * K
    moved = moved * 17 // 32 if op == "experts" else moved * 2
    return {"bytes": moved + rows * N * SIZE[case["out"]], "flops": 2 * rows * N * K}


# ---- inputs -------------------------------------------------------------------------------------

def _power2(e):
    """2^e in fp32 for whole e from -126 to 127, from the exponent field (a power function may be an ulp off)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _times_power2(v, e):
    """v·2^e in fp32, in two steps: either factor alone may leave the type's range."""
    half = torch.div(e, 2, rounding_mode="floor")
    return v * _power2(half) * _power2(e - half)


def _normal(gen, shape, dtype, sigma):
    return (torch.randn(shape, device="cuda", generator=gen) * sigma).to(dtype)


def _pack4(x):
    """A float matrix (..., K) as stored microscaled 4-bit data: codes (..., K/2), the lower nibble
    first, and scale bytes (..., K/32) at a row pitch of whole 16 bytes."""
    v = x.float().reshape(*x.shape[:-1], -1, BLOCK)
    amax = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = _times_power2(v.abs(), -e)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, edge in enumerate(edges):
        code += ((a >= edge) if i % 2 else (a > edge)).to(torch.uint8)
    code = (code | ((v < 0).to(torch.uint8) << 3)).reshape(*x.shape[:-1], -1)
    codes = (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous()
    s = (e + 127).to(torch.uint8).squeeze(-1)
    nb = s.shape[-1]
    held = torch.zeros(*s.shape[:-1], -(-nb // 16) * 16, dtype=torch.uint8, device=x.device)
    held[..., :nb] = s
    return codes, held[..., :nb]


def _split(case, seed):
    """Group borders: the active experts are drawn, each has a row, and the others fall by a skewed
    popularity, as a router's choices do."""
    rng = np.random.default_rng(seed)
    g, act, rows = case["groups"], case["active"], case["rows"]
    who = rng.permutation(g)[:act]
    pop = np.exp(0.7 * rng.standard_normal(act))
    sizes = np.zeros(g, dtype=np.int64)
    sizes[who] = 1 + rng.multinomial(rows - act, pop / pop.sum())
    return [0] + [int(v) for v in np.cumsum(sizes)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "quantize":
        # activations: a spread of magnitudes from row to row
        amp = torch.exp(torch.randn((case["rows"], 1), device="cuda", generator=gen))
        st["x"] = (torch.randn((case["rows"], case["cols"]), device="cuda", generator=gen) * amp).to(
            TORCH[case["dtype"]])
        return st
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        st["a"], st["as"] = _pack4(_normal(gen, (M, K), torch.float32, 1.0))
        st["b"], st["bs"] = _pack4(_normal(gen, (N, K), torch.float32, 0.02))
        return st
    st["borders"] = _split(case, seed)
    st["offsets"] = torch.tensor(st["borders"], dtype=torch.int32, device="cuda")
    total, g = case["rows"] + case["tail"], case["groups"]
    if op == "wgrad":
        dt = TORCH[case["dtype"]]
        st["x"] = _normal(gen, (total, case["P"]), dt, 1.0)
        st["y"] = _normal(gen, (total, case["Q"]), dt, 0.1)
        return st
    N, K = case["N"], case["K"]
    # the batch's buffer: rows behind the last group belong to the caller and stay as they are
    st["out"] = _normal(gen, (total, N), TORCH[case["out"]], 1.0)
    if op == "experts":
        st["a"], st["as"] = _pack4(_normal(gen, (total, K), torch.float32, 1.0))
        st["b"], st["bs"] = _pack4(_normal(gen, (g, N, K), torch.float32, 0.02))
        return st
    dt = TORCH[case["dtype"]]
    st["a"] = _normal(gen, (total, K), dt, 1.0)
    st["b"] = _normal(gen, (g, N, K) if case["layout"] == "nk" else (g, K, N), dt, 0.02)
    return st


# ---- one pass -----------------------------------------------------------------------------------

def _values4(codes, scales):
    """Values of stored microscaled 4-bit data, in fp32."""
    table = torch.tensor([*E2M1, *[-v for v in E2M1]], device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=-1)
    v = v.reshape(*codes.shape[:-1], -1, BLOCK)
    return _times_power2(v, scales.int()[..., None] - 127).reshape(*codes.shape[:-1], -1)


def _run_plain(st):
    op, case = st["op"], st["case"]
    if op == "quantize":
        x = st["x"].float()
        rows, cols = x.shape
        v = torch.zeros((rows, -(-cols // BLOCK) * BLOCK), device=x.device)
        v[:, :cols] = x
        v = v.reshape(rows, -1, BLOCK)
        amax = v.abs().amax(-1, keepdim=True)
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        a = _times_power2(v, -e)
        m = a.abs()
        step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
        q = (torch.round(m / step) * step).clamp(max=6.0) * torch.sign(a)
        return _times_power2(q, e).reshape(rows, -1)[:, :cols].to(TORCH[case["dtype"]])
    if op == "product":
        return torch.matmul(_values4(st["a"], st["as"]), _values4(st["b"], st["bs"]).t()).to(TORCH[case["out"]])
    edges = st["borders"]
    if op == "wgrad":
        out = torch.zeros((case["groups"], case["P"], case["Q"]), dtype=TORCH[case["out"]], device="cuda")
        for e in range(case["groups"]):
            if edges[e + 1] > edges[e]:
                x, y = st["x"][edges[e]:edges[e + 1]].float(), st["y"][edges[e]:edges[e + 1]].float()
                out[e] = torch.matmul(x.t(), y).to(out.dtype)
        return out
    out = st["out"]
    for e in range(case["groups"]):
        lo, hi = edges[e], edges[e + 1]
        if hi == lo:
            continue
        if op == "experts":
            a, b = _values4(st["a"][lo:hi], st["as"][lo:hi]), _values4(st["b"][e], st["bs"][e]).t()
        else:
            a, b = st["a"][lo:hi].float(), st["b"][e].float()
            b = b.t() if case["layout"] == "nk" else b
        out[lo:hi] = torch.matmul(a, b).to(out.dtype)
    return out


def _run_own(st):
    from tiled_bf16_gemm_amd import torch_ops
    op, case = st["op"], st["case"]
    if op == "quantize":
        codes, scales = torch_ops.mx4_quantize(st["x"])
        return torch_ops.mx4_dequantize(codes, scales, cols=case["cols"], out_dtype=case["dtype"])
    if op == "product":
        return torch_ops.mx4_gemm(st["a"], st["as"], st["b"], st["bs"], out_dtype=case["out"])
    if op == "wgrad":
        return torch_ops.gemm_grouped_wgrad(st["x"], st["y"], st["offsets"], out_dtype=case["out"])
    if op == "experts":
        return torch_ops.mx4_gemm_grouped(st["a"], st["as"], st["b"], st["bs"], st["offsets"], out_dtype=case["out"],
                                          out=st["out"])
    return torch_ops.gemm_grouped(st["a"], st["b"], st["offsets"], b_layout=case["layout"], out_dtype=case["out"],
                                  out=st["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits ------------------------------------------------------------------

def _double_power2(e):
    """2^e in fp64 for whole e, from the exponent field."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _decode64(codes, scales):
    """Microscaled values from the format's fields: sign, two exponent bits, one mantissa bit."""
    c = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.int64, device=codes.device)
    c[..., 0::2] = codes.long() % 16
    c[..., 1::2] = codes.long() // 16
    sign = 1.0 - 2.0 * (c // 8).double()
    ex, mant = (c // 2) % 4, (c % 2).double()
    mag = torch.where(ex == 0, mant / 2, (1 + mant / 2) * _double_power2(ex - 1))
    return sign * mag * _double_power2(scales.long() - 127).repeat_interleave(BLOCK, dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    op = st["op"]
    if op == "quantize":
        x = st["x"].double()
        rows, cols = x.shape
        out = torch.empty_like(x)
        for lo in range(0, cols, BLOCK):
            v = x[:, lo:lo + BLOCK]
            top = v.abs().amax(1, keepdim=True)
            e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
            # log2 may round across a power of two: settle it by comparison
            e = torch.where(_double_power2(e) > top, e - 1, e)
            e = torch.where(_double_power2(e + 1) <= top, e + 1, e)
            scale = _double_power2(torch.clamp(e - 2, -127, 127))
            m = v.abs() / scale
            q = torch.zeros_like(m)
            for i in range(1, 8):
                mid = (E2M1[i - 1] + E2M1[i]) / 2
                q = torch.where((m >= mid) if i % 2 == 0 else (m > mid), torch.full_like(m, E2M1[i]), q)
            out[:, lo:lo + BLOCK] = torch.where(top > 0, torch.copysign(q * scale, v), torch.zeros_like(v))
        return out
    if op == "product":
        return _decode64(st["a"], st["as"]) @ _decode64(st["b"], st["bs"]).t().contiguous()
    edges = st["borders"]
    spans = [(e, slice(edges[e], edges[e + 1])) for e in range(case["groups"])]
    if op == "wgrad":
        return torch.stack([st["x"][s].double().t().contiguous() @ st["y"][s].double() for _, s in spans])
    out = st["out"].double()
    for e, s in spans:
        if op == "experts":
            out[s] = _decode64(st["a"][s], st["as"][s]) @ _decode64(st["b"][e], st["bs"][e]).t().contiguous()
        else:
            b = st["b"][e].double()
            out[s] = st["a"][s].double() @ (b.t().contiguous() if case["layout"] == "nk" else b)
    return out
