"""Measured cases of what stands around the products of expert layers, and of weights in 4 bits.

Six operators, each with its plain form in elementary torch operations and the call a user's
program makes of this package:

  sort          a router's choices -> groups of rows: offsets, the slot of every row, the row of every slot
  dispatch      rows[place[t, j]] = X[t]: the tokens' rows, copied to their experts' groups
  combine       out[t] = sum over j of w[t, j]·Y[place[t, j]]: the experts' rows back to their tokens
                (without w: the gradient of X under dispatch)
  combine_grad  the gradients of Y and of w under combine
  w4            C = A·Wᵀ with W in whole 4-bit codes, a scale (and a zero) for every group of the sum's index
  w4_experts    w4 over ragged groups with a W each; rows of A taken through the sort or in order

A case is a dict of plain values; prepare() draws its inputs from the seed alone, run() makes one
pass, exact() gives the definition's value in 64 bits, work() the bytes and operations that a pass
cannot do without.  `own` is False for the plain forms and True for the package's kernels.
"""
import math

import torch

own = False

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---- cases --------------------------------------------------------------------------------------

def listed():
    return [
        # one decoding step: 8 tokens, 8 experts each, of 64: launch latency counts
        dict(name="sort_8x8_64e", op="sort", tokens=8, top_k=8, groups=64, active=40, pad=0),
        # a long prefill or training batch with padded tokens
        dict(name="sort_16384x8_256e", op="sort", tokens=16384, top_k=8, groups=256, active=256, pad=191),
        # a short, odd batch: rows of an odd length, padded
        dict(name="dispatch_777x2049_f16", op="dispatch", tokens=777, top_k=3, groups=31, active=29, pad=23, H=2049,
             dtype="f16"),
        # a training step's rows of two experts each
        dict(name="dispatch_8192x4096_bf16", op="dispatch", tokens=8192, top_k=2, groups=8, active=8, pad=0, H=4096,
             dtype="bf16"),
        # the decoding step's way back
        dict(name="combine_8x8x4096_bf16", op="combine", tokens=8, top_k=8, groups=64, active=40, pad=0, H=4096,
             dtype="bf16", out="bf16", weighted=True),
        # the way back of many small experts
        dict(name="combine_8192x8x4096_bf16", op="combine", tokens=8192, top_k=8, groups=128, active=128, pad=0,
             H=4096, dtype="bf16", out="bf16", weighted=True),
        # gradients of an odd, padded batch
        dict(name="combine_grad_2047x1001_f16", op="combine_grad", tokens=2047, top_k=4, groups=32, active=31, pad=64,
             H=1001, dtype="f16", out="f16"),
        # gradients of a training step
        dict(name="combine_grad_8192x4096_bf16", op="combine_grad", tokens=8192, top_k=2, groups=8, active=8, pad=0,
             H=4096, dtype="bf16", out="bf16"),
        # one token through a wide layer
        dict(name="w4_1x14336x4096", op="w4", M=1, N=14336, K=4096, group=128, zeros=False, dtype="bf16", out="bf16"),
        # a batch of requests, short groups with zeros, sizes off every tile
        dict(name="w4_33x2049x8160_f16", op="w4", M=33, N=2049, K=8160, group=32, zeros=True, dtype="f16", out="f32"),
        # decoding: 8 tokens through 8 experts each, their rows read through the sort
        dict(name="w4_experts_decode_64e", op="w4_experts", tokens=8, top_k=8, groups=64, active=40, pad=0, N=4096,
             K=2048, group=128, zeros=False, dtype="bf16", out="bf16", gather=True),
        # a larger batch of requests, rows already sorted
        dict(name="w4_experts_2048_64e", op="w4_experts", tokens=256, top_k=8, groups=64, active=64, pad=5, N=2048,
             K=4096, group=64, zeros=True, dtype="bf16", out="bf16", gather=False),
    ]


def _spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _routing(rng, most, experts):
    """Tokens, choices, experts and padding of a batch of up to `most` tokens."""
    groups = _spread(rng, 2, experts)
    top_k = rng.randint(1, min(8, groups))
    tokens = _spread(rng, 1, most)
    pad = rng.choice([0, 0, rng.randint(0, tokens // 4)])
    active = rng.randint(max(top_k, groups // 2), groups)
    return dict(tokens=tokens, top_k=top_k, groups=groups, pad=pad, active=max(top_k, min(active, (tokens - pad) * top_k)))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "combine_grad", "w4", "w4_experts"])
    if op == "sort":
        return dict(op=op, **_routing(rng, 16384, 256))
    if op == "w4":
        group = rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "f16"])
        return dict(op=op, M=_spread(rng, 1, 256), N=_spread(rng, 16, 14336), K=group * _spread(rng, 1, 8192 // group),
                    group=group, zeros=rng.random() < 0.5, dtype=dtype, out=rng.choice([dtype, "f32"]))
    if op == "w4_experts":
        group = rng.choice([32, 64, 128])
        dtype = rng.choice(["bf16", "f16"])
        return dict(op=op, **_routing(rng, 256, 64), N=_spread(rng, 16, 2048), K=group * _spread(rng, 1, 4096 // group),
                    group=group, zeros=rng.random() < 0.5, dtype=dtype, out=rng.choice([dtype, "f32"]),
                    gather=rng.random() < 0.5)
    case = dict(op=op, **_routing(rng, 8192, 128), H=_spread(rng, 16, 8192), dtype=rng.choice(["bf16", "f16", "f32"]))
    while case["tokens"] * case["top_k"] * case["H"] * SIZE[case["dtype"]] > 8192 * 2 * 4096 * 2:
        case["H"] = max(16, case["H"] // 2)
    if op != "dispatch":
        case["out"] = rng.choice(["f32", case["dtype"]])
    if op == "combine":
        case["weighted"] = rng.random() < 0.75
    return case


def work(case):
    op = case["op"]
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        weights = N * K // 2 + N * (K // case["group"]) * (3 if case["zeros"] else 2)
        return {"bytes": weights + M * K * 2 + M * N * SIZE[case["out"]], "flops": 2 * M * N * K}
    T, k = case["tokens"], case["top_k"]
    n, used = T * k, (T - case["pad"]) * k
    if op == "sort":
        return {"bytes": 12 * n + 4 * (case["groups"] + 1), "flops": n}
    if op == "w4_experts":
        N, K = case["N"], case["K"]
        weights = N * K // 2 + N * (K // case["group"]) * (3 if case["zeros"] else 2)
        rows = T - case["pad"] if case["gather"] else used
        return {"bytes": case["active"] * weights + rows * K * 2 + used * N * SIZE[case["out"]] + 4 * used * case["gather"],
                "flops": 2 * used * N * K}
    H, b = case["H"], SIZE[case["dtype"]]
    if op == "dispatch":
        return {"bytes": (T - case["pad"] + used) * H * b + 4 * n, "flops": 0}
    bo = SIZE[case["out"]]
    if op == "combine":
        return {"bytes": used * H * b + T * H * bo + (8 if case["weighted"] else 4) * n, "flops": 2 * used * H}
    return {"bytes": (T - case["pad"]) * H * bo + 2 * used * H * b + 12 * n, "flops": 3 * used * H}


# ---- inputs -------------------------------------------------------------------------------------

def _normal(gen, shape, dtype, sigma):
    return (torch.randn(shape, device="cuda", generator=gen) * sigma).to(dtype)


def _choices(case, gen):
    """A router's choices, (tokens, top_k) int32: `active` of the experts by a skewed popularity, each taken
    by a token at least, no expert twice for a token; padded tokens (the last ones) hold -1."""
    T, k, E, act = case["tokens"], case["top_k"], case["groups"], case["active"]
    who = torch.randperm(E, device="cuda", generator=gen)[:act]
    score = torch.randn((T, act), device="cuda", generator=gen) + 0.7 * torch.randn(act, device="cuda", generator=gen)
    slots = torch.arange(-(-act // k) * k, device="cuda")
    score[slots // k, slots % act] += 100.0
    ids = who[score.topk(k, dim=1).indices].to(torch.int32)
    ids[T - case["pad"]:] = -1
    return ids.contiguous()


def _sorted_by_expert(ids, groups):
    """offsets, source and place of a router's choices."""
    flat = ids.flatten().long()
    n = flat.numel()
    key = torch.where((flat >= 0) & (flat < groups), flat, groups)
    ordered, slot = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(groups + 1, device=flat.device)).to(torch.int32)
    row = torch.arange(n, device=flat.device)
    held = ordered < groups
    source = torch.where(held, slot, -1).to(torch.int32)
    place = torch.empty(n, dtype=torch.int32, device=flat.device)
    place[slot] = torch.where(held, row, -1).to(torch.int32)
    return offsets, source, place.reshape(ids.shape)


def _quantized(gen, N, K, group, zeros, dtype):
    """Weights of a layer in whole 4-bit codes: (codes (N, K/2), the lower nibble first, scales and zeros (K/group, N))."""
    w = (torch.randn((N, K // group, group), device="cuda", generator=gen) * 0.02)
    if zeros:
        lo, hi = w.amin(-1), w.amax(-1)
        scale = ((hi - lo) / 15).to(dtype)
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
    else:
        scale = (w.abs().amax(-1) / 7).to(dtype)
        zero = torch.full_like(scale, 8.0, dtype=torch.float32)
    code = (torch.round(w / scale.float()[..., None]) + zero[..., None]).clamp(0, 15).to(torch.uint8).reshape(N, K)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    return codes, scale.t().contiguous(), zero.to(torch.uint8).t().contiguous() if zeros else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        dt = TORCH[case["dtype"]]
        st["a"] = _normal(gen, (M, K), dt, 1.0)
        codes, st["scales"], st["zeros"] = _quantized(gen, N, K, case["group"], case["zeros"], dt)
        # rows of codes on 16 bytes
        pitch = -(-K // 32) * 16
        st["codes"] = torch.zeros((N, pitch), dtype=torch.uint8, device="cuda")[:, :K // 2]
        st["codes"].copy_(codes)
        return st
    ids = _choices(case, gen)
    if op == "sort":
        st["experts"] = ids
        return st
    st["offsets"], st["source"], st["place"] = _sorted_by_expert(ids, case["groups"])
    T, k = case["tokens"], case["top_k"]
    rows = T * k
    if op == "w4_experts":
        N, K, E = case["N"], case["K"], case["groups"]
        dt = TORCH[case["dtype"]]
        st["borders"] = st["offsets"].tolist()
        st["a"] = _normal(gen, (T if case["gather"] else rows, K), dt, 1.0)
        # the batch's buffer: rows behind the last group belong to the caller and stay as they are
        st["out"] = _normal(gen, (rows, N), TORCH[case["out"]], 1.0)
        parts = [_quantized(gen, N, K, case["group"], case["zeros"], dt) for _ in range(E)]
        pitch = -(-K // 32) * 16
        st["codes"] = torch.zeros((E, N, pitch), dtype=torch.uint8, device="cuda")[:, :, :K // 2]
        st["codes"].copy_(torch.stack([p[0] for p in parts]))
        st["scales"] = torch.stack([p[1] for p in parts])
        st["zeros"] = torch.stack([p[2] for p in parts]) if case["zeros"] else None
        return st
    H, dt = case["H"], TORCH[case["dtype"]]
    if op == "dispatch":
        st["x"] = _normal(gen, (T, H), dt, 1.0)
        st["out"] = _normal(gen, (rows, H), dt, 1.0)
        return st
    st["y"] = _normal(gen, (rows, H), dt, 1.0)
    st["w"] = torch.softmax(torch.randn((T, k), device="cuda", generator=gen), dim=1)
    if op == "combine_grad":
        st["dout"] = _normal(gen, (T, H), TORCH[case["out"]], 0.1)
        st["dy"] = _normal(gen, (rows, H), dt, 1.0)
    return st


# ---- one pass -----------------------------------------------------------------------------------

def _weights(codes, scales, zeros):
    """The values of a 4-bit matrix, (N, K) fp32 (a 16-bit scale times a whole number below 2^8 is exact there)."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(1).float().reshape(codes.shape[0], scales.shape[0], -1)
    z = 8.0 if zeros is None else zeros.t().float()[..., None]
    return ((c - z) * scales.t().float()[..., None]).flatten(1)


def _run_plain(st):
    op, case = st["op"], st["case"]
    if op == "w4":
        return (st["a"].float() @ _weights(st["codes"], st["scales"], st["zeros"]).t()).to(TORCH[case["out"]])
    if op == "sort":
        return _sorted_by_expert(st["experts"], case["groups"])
    if op == "w4_experts":
        out, edges = st["out"], st["borders"]
        for e in range(case["groups"]):
            lo, hi = edges[e], edges[e + 1]
            if hi > lo:
                a = st["a"][(st["source"][lo:hi] // case["top_k"]).long()] if case["gather"] else st["a"][lo:hi]
                w = _weights(st["codes"][e], st["scales"][e], None if st["zeros"] is None else st["zeros"][e])
                out[lo:hi] = (a.float() @ w.t()).to(out.dtype)
        return out
    place = st["place"].long()
    held = place >= 0
    if op == "dispatch":
        token, _ = torch.nonzero(held, as_tuple=True)
        st["out"][place[held]] = st["x"][token]
        return st["out"]
    at = place.clamp(min=0)
    if op == "combine":
        w = st["w"] * held if case["weighted"] else held.float()
        return (w[..., None] * st["y"][at].float()).sum(1).to(TORCH[case["out"]])
    dout = st["dout"].float()
    token, _ = torch.nonzero(held, as_tuple=True)
    st["dy"][place[held]] = (st["w"][held][:, None] * dout[token]).to(st["dy"].dtype)
    return st["dy"], (st["y"][at].float() * dout[:, None]).sum(-1) * held


def _run_own(st):
    from tiled_bf16_gemm_amd import torch_ops
    op, case = st["op"], st["case"]
    if op == "w4":
        return torch_ops.w4_gemm(st["a"], st["codes"], st["scales"], st["zeros"], out_dtype=case["out"])
    if op == "sort":
        return torch_ops.expert_sort(st["experts"], case["groups"])
    if op == "w4_experts":
        return torch_ops.w4_gemm_grouped(st["a"], st["codes"], st["scales"], st["offsets"], st["zeros"],
                                         source=st["source"] if case["gather"] else None, top_k=case["top_k"],
                                         out_dtype=case["out"], out=st["out"])
    if op == "dispatch":
        return torch_ops.expert_dispatch(st["x"], st["place"], out=st["out"])
    if op == "combine":
        return torch_ops.expert_combine(st["y"], st["place"], st["w"] if case["weighted"] else None,
                                        out_dtype=case["out"])
    return torch_ops.expert_combine_grad(st["dout"], st["y"], st["place"], st["w"], dy=st["dy"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits ------------------------------------------------------------------

def _weights64(codes, scales, zeros):
    N, half = codes.shape
    w = torch.empty((N, 2 * half), dtype=torch.float64, device=codes.device)
    w[:, 0::2] = (codes.long() % 16).double()
    w[:, 1::2] = (codes.long() // 16).double()
    groups = scales.shape[0]
    per = 2 * half // groups
    for g in range(groups):
        z = 8.0 if zeros is None else zeros[g].double()[:, None]
        w[:, g * per:(g + 1) * per] = scales[g].double()[:, None] * (w[:, g * per:(g + 1) * per] - z)
    return w


def exact(case, seed):
    op = case["op"]
    if op == "sort":
        return None
    st = prepare(case, seed)
    if op == "w4":
        return st["a"].double() @ _weights64(st["codes"], st["scales"], st["zeros"]).t().contiguous()
    source, k = st["source"].long(), case["top_k"]
    filled = int(st["offsets"][-1])
    slot = source[:filled]
    token = slot // k
    if op == "w4_experts":
        out, edges = st["out"].double(), st["borders"]
        for e in range(case["groups"]):
            s = slice(edges[e], edges[e + 1])
            if s.stop > s.start:
                a = st["a"][token[s]] if case["gather"] else st["a"][s]
                out[s] = a.double() @ _weights64(st["codes"][e], st["scales"][e],
                                                 None if st["zeros"] is None else st["zeros"][e]).t().contiguous()
        return out
    if op == "dispatch":
        out = st["out"].double()
        out[:filled] = st["x"].double()[token]
        return out
    w = st["w"].double().flatten()[slot]
    y = st["y"][:filled].double()
    if op == "combine":
        out = torch.zeros((case["tokens"], case["H"]), dtype=torch.float64, device="cuda")
        return out.index_add_(0, token, w[:, None] * y if case["weighted"] else y)
    dout = st["dout"].double()[token]
    dy = st["dy"].double()
    dy[:filled] = w[:, None] * dout
    dw = torch.zeros(case["tokens"] * k, dtype=torch.float64, device="cuda")
    dw[slot] = (y * dout).sum(1)
    return dy, dw.reshape(case["tokens"], k)
