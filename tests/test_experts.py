"""Tokens sorted by expert, their rows to the groups and back, and the gradients (tbg_expert_sort,
tbg_expert_dispatch, tbg_expert_combine, tbg_expert_combine_grad).

Sorting and copying are exact.  Combining is an fp32 sum of top_k products, each step off by at most half
a unit in the last place of a partial sum (2^-24 relative to the sum of magnitudes), then rounded once:
|out - exact| <= (k + 1)·2^-23·sum|w·y| + eps/2·(|exact| + that).  dY is one fp32 product rounded to its
type, the same two roundings torch makes.  dweights is an fp32 sum of `cols` products in some order:
|dw - exact| <= (cols + 1)·2^-23·sum|y·d|."""
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

def _sort_args(**over):
    a = dict(slots=64, groups=8, experts=PTR, offsets=PTR, source=PTR, place=PTR)
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(slots=-1), tbg.ERR_INVALID_VALUE),
    (dict(groups=-1), tbg.ERR_INVALID_VALUE),
    (dict(slots=(1 << 30) + 1), tbg.ERR_UNSUPPORTED),
    (dict(groups=4097), tbg.ERR_UNSUPPORTED),
    (dict(experts=0), tbg.ERR_INVALID_VALUE),
    (dict(offsets=0), tbg.ERR_INVALID_VALUE),
    (dict(offsets=0, slots=0), tbg.ERR_INVALID_VALUE),
    (dict(source=0), tbg.ERR_INVALID_VALUE),
    (dict(place=0), tbg.ERR_INVALID_VALUE),
    (dict(experts=PTR + 2), tbg.ERR_MISALIGNED),
    (dict(offsets=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(source=PTR + 2), tbg.ERR_MISALIGNED),
    (dict(place=PTR + 3), tbg.ERR_MISALIGNED),
    (dict(slots=100000), tbg.ERR_OUT_OF_RANGE),
    (dict(slots=100000, workspace=PTR, workspace_bytes=64), tbg.ERR_OUT_OF_RANGE),
    (dict(slots=100000, workspace=PTR + 16, workspace_bytes=1 << 20), tbg.ERR_MISALIGNED),
])
def test_sort_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.expert_sort(**_sort_args(**over))
    assert e.value.status == status, e.value


def _dispatch_args(**over):
    a = dict(tokens=8, top_k=2, rows=16, cols=24, dtype="bf16", X=PTR, ldx=24, place=PTR, out=PTR, ld_out=24)
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), tbg.ERR_INVALID_VALUE),
    (dict(top_k=-1), tbg.ERR_INVALID_VALUE),
    (dict(rows=-1), tbg.ERR_INVALID_VALUE),
    (dict(cols=-1), tbg.ERR_INVALID_VALUE),
    (dict(top_k=1025), tbg.ERR_UNSUPPORTED),
    (dict(tokens=1 << 30, top_k=2), tbg.ERR_UNSUPPORTED),
    (dict(tokens=(1 << 30) + 1, top_k=0), tbg.ERR_UNSUPPORTED),
    (dict(rows=(1 << 30) + 1), tbg.ERR_UNSUPPORTED),
    (dict(cols=(1 << 30) + 1, ldx=1 << 31, ld_out=1 << 31), tbg.ERR_UNSUPPORTED),
    (dict(dtype=8), tbg.ERR_INVALID_VALUE),
    (dict(X=0), tbg.ERR_INVALID_VALUE),
    (dict(X=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(out=0), tbg.ERR_INVALID_VALUE),
    (dict(out=PTR + 2, dtype="f32"), tbg.ERR_MISALIGNED),
    (dict(ldx=23), tbg.ERR_INVALID_VALUE),
    (dict(ld_out=23), tbg.ERR_INVALID_VALUE),
    (dict(ld_out=(1 << 40) + 1), tbg.ERR_UNSUPPORTED),
    (dict(place=0), tbg.ERR_INVALID_VALUE),
    (dict(place=PTR + 2), tbg.ERR_MISALIGNED),
])
def test_dispatch_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.expert_dispatch(**_dispatch_args(**over))
    assert e.value.status == status, e.value


def _combine_args(**over):
    a = dict(tokens=8, top_k=2, rows=16, cols=24, Y=PTR, ldy=24, y_dtype="bf16", place=PTR, weights=PTR, out=PTR,
             ld_out=24, out_dtype="bf16")
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), tbg.ERR_INVALID_VALUE),
    (dict(top_k=1025), tbg.ERR_UNSUPPORTED),
    (dict(y_dtype="u16"), tbg.ERR_INVALID_VALUE),
    (dict(out_dtype="f16"), tbg.ERR_INVALID_VALUE),
    (dict(y_dtype="f32"), tbg.ERR_INVALID_VALUE),  # out bf16 of an fp32 Y
    (dict(Y=0), tbg.ERR_INVALID_VALUE),
    (dict(Y=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(out=0), tbg.ERR_INVALID_VALUE),
    (dict(out=PTR + 2, out_dtype="f32"), tbg.ERR_MISALIGNED),
    (dict(ldy=23), tbg.ERR_INVALID_VALUE),
    (dict(ld_out=23), tbg.ERR_INVALID_VALUE),
    (dict(place=0), tbg.ERR_INVALID_VALUE),
    (dict(weights=PTR + 2), tbg.ERR_MISALIGNED),
])
def test_combine_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.expert_combine(**_combine_args(**over))
    assert e.value.status == status, e.value


def _grad_args(**over):
    a = dict(tokens=8, top_k=2, rows=16, cols=24, dout=PTR, ldd=24, dout_dtype="f32", Y=PTR, ldy=24, y_dtype="bf16",
             place=PTR, weights=PTR, dY=PTR, ld_dy=24, dweights=PTR)
    a.update(over)
    return a


@pytest.mark.parametrize("over,status", [
    (dict(cols=-1), tbg.ERR_INVALID_VALUE),
    (dict(top_k=1025), tbg.ERR_UNSUPPORTED),
    (dict(dout_dtype="f16"), tbg.ERR_INVALID_VALUE),
    (dict(y_dtype="u8"), tbg.ERR_INVALID_VALUE),
    (dict(dout=0), tbg.ERR_INVALID_VALUE),
    (dict(dout=PTR + 2), tbg.ERR_MISALIGNED),
    (dict(Y=0), tbg.ERR_INVALID_VALUE),
    (dict(dY=0), tbg.ERR_INVALID_VALUE),
    (dict(dY=PTR + 1), tbg.ERR_MISALIGNED),
    (dict(ldd=23), tbg.ERR_INVALID_VALUE),
    (dict(ldy=23), tbg.ERR_INVALID_VALUE),
    (dict(ld_dy=23), tbg.ERR_INVALID_VALUE),
    (dict(place=0), tbg.ERR_INVALID_VALUE),
    (dict(dweights=0), tbg.ERR_INVALID_VALUE),
    (dict(dweights=PTR + 2), tbg.ERR_MISALIGNED),
])
def test_combine_grad_refusals(over, status):
    with pytest.raises(tbg.Error) as e:
        tbg.expert_combine_grad(**_grad_args(**over))
    assert e.value.status == status, e.value


def test_no_ops_need_no_device():
    tbg.expert_dispatch(**_dispatch_args(tokens=0, X=0, place=0))
    tbg.expert_dispatch(**_dispatch_args(rows=0, out=0))
    tbg.expert_dispatch(**_dispatch_args(cols=0, X=0, out=0))
    tbg.expert_combine(**_combine_args(tokens=0, out=0, place=0))
    tbg.expert_combine(**_combine_args(cols=0, out=0, Y=0))
    tbg.expert_combine_grad(**_grad_args(tokens=0, dout=0, place=0, dweights=0))
    tbg.expert_combine_grad(**_grad_args(top_k=0, place=0, dweights=0))


def test_sort_workspace():
    assert tbg.expert_sort_workspace_query(0, 8) == tbg.expert_sort_workspace_query(4096, 512) == 0
    assert tbg.expert_sort_workspace_query(-1, 8) == tbg.expert_sort_workspace_query(8, 4097) == 0
    for slots in (4097, 100000, 1 << 24, 1 << 30):
        for groups in (1, 8, 256, 4096):
            need = tbg.expert_sort_workspace_query(slots, groups)
            assert 0 < need <= 256 * groups * 4 + 256 and need % 256 == 0


def test_helpers_refuse():
    ops = _ops()
    ids, x = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 8))
    for call in (lambda: ops.expert_sort(ids, 4), lambda: ops.expert_dispatch(x, ids), lambda: ops.expert_combine(x, ids),
                 lambda: ops.expert_combine_grad(x, x, ids)):
        with pytest.raises(ValueError):  # host tensors
            call()


# ---- sorting ----------------------------------------------------------------------------------------

def _sorted(ids, groups):
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(groups + 1))
    source = np.where(key[order] < groups, order, -1)
    place = np.full(flat.size, -1)
    place[order] = np.where(key[order] < groups, np.arange(flat.size), -1)
    return offsets.astype(np.int32), source.astype(np.int32), place.astype(np.int32).reshape(ids.shape)


def _check_sort(ids, groups, got):
    for name, g, w in zip(("offsets", "source", "place"), got, _sorted(ids, groups)):
        assert np.array_equal(g.cpu().numpy(), w), (name, ids.size, groups)


SORTS = [(1, 1), (1, 4096), (63, 5), (64, 64), (65, 2), (1000, 1), (1024, 256), (1025, 7), (4096, 512), (4097, 512),
         (512, 4096), (513, 4096), (2049, 1024), (3000, 4096), (20000, 3), (131072, 256), (300001, 130), (700000, 4096)]


@gpu
@pytest.mark.parametrize("slots,groups", SORTS)
def test_sort(slots, groups):
    print(f"sort {slots} slots, {groups} groups", flush=True)
    rng = np.random.default_rng(slots + groups)
    for kind in range(3):
        ids = rng.integers(0, groups, slots)
        if kind == 1:  # a few popular experts, and slots of no expert
            ids = np.minimum(ids, rng.integers(0, groups, slots))
            ids[rng.random(slots) < 0.2] = rng.choice([-1, groups, groups + 1, -2 ** 31, 2 ** 31 - 1])
        if kind == 2:  # one expert has all
            ids[:] = groups - 1
        ids = ids.astype(np.int32)
        _check_sort(ids, groups, _ops().expert_sort(torch.from_numpy(ids).cuda(), groups))


@gpu
def test_sort_of_nothing():
    ops = _ops()
    off, src, place = ops.expert_sort(torch.zeros((0, 4), dtype=torch.int32, device="cuda"), 9)
    assert off.tolist() == [0] * 10 and src.numel() == 0 and place.shape == (0, 4)
    for n in (5, 5000):  # no experts at all
        off, src, place = ops.expert_sort(torch.arange(n, dtype=torch.int32, device="cuda"), 0)
        assert off.tolist() == [0] and bool((src == -1).all()) and bool((place == -1).all())


@gpu
def test_sort_writes_nothing_else():
    for slots, groups in ((70, 9), (9000, 33)):
        ids = torch.randint(0, groups, (slots,), dtype=torch.int32, device="cuda")
        bufs = [torch.full((n + 16,), 77, dtype=torch.int32, device="cuda") for n in (groups + 1, slots, slots)]
        need = tbg.expert_sort_workspace_query(slots, groups)
        ws = torch.full((need + 256,), 5, dtype=torch.uint8, device="cuda")
        tbg.expert_sort(slots, groups, ids.data_ptr(), *[b.data_ptr() + 32 for b in bufs], ws.data_ptr(), need,
                        torch.cuda.current_stream().cuda_stream)
        got = [b[8:-8] for b in bufs]
        _check_sort(ids.cpu().numpy(), groups, got)
        assert all(bool((b[:8] == 77).all()) and bool((b[-8:] == 77).all()) for b in bufs)
        assert bool((ws[need:] == 5).all())


# ---- rows to the groups -----------------------------------------------------------------------------

def _routing(T, k, E, seed, drop=0.1):
    """Distinct experts for every token, some slots dropped, and their sort."""
    rng = np.random.default_rng(seed)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    ids[rng.random((T, k)) < drop] = -1
    off, src, place = _sorted(ids, E)
    return [torch.from_numpy(a).cuda() for a in (off, src, place)]


def _padded(t, ld, fill):
    full = torch.full((t.shape[0], ld), fill, dtype=t.dtype, device=t.device)
    full[:, :t.shape[1]] = t
    return full[:, :t.shape[1]]


def _bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


@gpu
@pytest.mark.parametrize("dtype", [torch.uint8, torch.bfloat16, torch.float16, torch.float32, torch.int32])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (3, 2, 4, 7), (5, 3, 8, 16), (9, 8, 8, 33), (40, 1, 3, 17), (7, 4, 64, 2049),
                                     (65, 2, 8, 130)])
def test_dispatch(T, k, E, H, dtype):
    print(f"dispatch {T}x{k} of {E}, {H} {dtype}", flush=True)
    _, src, place = _routing(T, k, E, T * 31 + H)
    x = (torch.randint(-100, 100, (T, H), device="cuda", generator=_gen(H))).to(dtype)
    want = torch.full((T * k, H), 9, device="cuda").to(dtype)
    n = int((src >= 0).sum())
    want[:n] = x[(src[:n] // k).long()]
    for pad in (0, 5):
        out = torch.full((T * k + 2, H + pad), 9, device="cuda").to(dtype)
        got = _ops().expert_dispatch(_padded(x, H + 3 * pad, 1) if pad else x, place, out=out[1:-1, :H] if pad else out[1:-1])
        assert torch.equal(_bits(got), _bits(want))
        assert bool((out[0] == 9).all()) and bool((out[-1] == 9).all()) and bool((out[:, H:] == 9).all())


@gpu
def test_dispatch_keeps_bits_of_nan():
    x = torch.tensor([[0x7F81, -1, 0x7FC1, 0x0001] * 5], dtype=torch.int16, device="cuda").view(torch.bfloat16)
    place = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    out = _ops().expert_dispatch(x, place)
    assert torch.equal(_bits(out[0]), _bits(x[0])) and torch.equal(_bits(out[1]), _bits(x[0]))


@gpu
def test_rows_outside_are_no_rows():
    """Values of place outside the rows, whatever they are, touch nothing."""
    ops = _ops()
    bad = [-1, -2 ** 31, 4, 2 ** 31 - 1]
    place = torch.tensor([[0, bad[0]], [bad[1], bad[2]], [3, bad[3]]], dtype=torch.int32, device="cuda")
    x = torch.arange(1, 61, dtype=torch.float32, device="cuda").reshape(3, 20)
    out = torch.zeros((4, 20), device="cuda")
    ops.expert_dispatch(x, place, out=out)
    assert torch.equal(out, torch.stack([x[0], out[1] * 0, out[1] * 0, x[2]]))
    w = torch.full((3, 2), 2.0, device="cuda")
    w[0, 1] = w[1, 0] = float("nan")  # the weight of no row does not count
    got = ops.expert_combine(out, place, w)
    assert torch.equal(got, torch.stack([2 * x[0], x[0] * 0, 2 * x[2]]))
    dy, dw = ops.expert_combine_grad(x, out, place, w, dy=torch.zeros((4, 20), device="cuda"))
    assert torch.equal(dy, torch.stack([2 * x[0], x[0] * 0, x[0] * 0, 2 * x[2]]))
    want = torch.stack([(x[0] * x[0]).sum(), x[0, 0] * 0, x[0, 0] * 0, x[0, 0] * 0, (x[2] * x[2]).sum(), x[0, 0] * 0])
    assert torch.equal(dw.flatten(), want)  # whole numbers below 2^24


@gpu
@pytest.mark.parametrize("top_k,cols", [(2, 5), (4, 20), (9, 1501)])
def test_slots_that_hold_the_same_row(top_k, cols):
    """Of slots that hold one row, every element is one of theirs; combine and dweights count each slot."""
    ops = _ops()
    tokens = 6
    x = torch.randint(1, 9, (tokens, cols), generator=_gen(3), device="cuda").float()
    place = (torch.arange(tokens * top_k, dtype=torch.int32, device="cuda") % 4).reshape(tokens, top_k).contiguous()
    w = torch.randint(1, 9, (tokens, top_k), generator=_gen(4), device="cuda").float()
    out = ops.expert_dispatch(x, place, out=torch.full((5, cols), -1.0, device="cuda"))
    dy, dw = ops.expert_combine_grad(x, out, place, w, dy=torch.full((5, cols), -1.0, device="cuda"))
    for row in range(4):
        t, j = (place == row).nonzero(as_tuple=True)
        assert bool((out[row] == x[t]).any(dim=0).all())
        assert bool((dy[row] == w[t, j, None] * x[t]).any(dim=0).all())
    assert bool((out[4] == -1).all()) and bool((dy[4] == -1).all())
    # whole numbers: at most 1501 * 64 and 9 * 64, which fp32 holds
    assert torch.equal(dw, (out[place.long()] * x[:, None]).sum(-1))
    assert torch.equal(ops.expert_combine(out, place, w), (w[..., None] * out[place.long()]).sum(1))


# ---- rows back to their tokens ----------------------------------------------------------------------

def _combine64(y, place, w):
    T, k = place.shape
    out = torch.zeros((T, y.shape[1]), dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(out)
    for j in range(k):
        held = place[:, j] >= 0
        term = y[place[held, j].long()].double() * (w[held, j].double()[:, None] if w is not None else 1.0)
        out[held] += term
        mag[held] += term.abs()
    return out, mag


@gpu
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (3, 2, 4, 3), (5, 3, 8, 8), (9, 8, 8, 33), (4, 9, 16, 40), (7, 5, 64, 2049),
                                     (65, 2, 8, 130), (2, 17, 32, 12)])
def test_combine(T, k, E, H, dtype, out):
    print(f"combine {T}x{k} of {E}, {H} {dtype} -> {out}", flush=True)
    _, _, place = _routing(T, k, E, T * 7 + H)
    place[T - 1] = -1  # a token without a row
    y = torch.randn((T * k, H), device="cuda", generator=_gen(H)).to(TORCH[dtype])
    w = torch.randn((T, k), device="cuda", generator=_gen(H + 1))
    eps = torch.finfo(TORCH[out]).eps / 2
    for weights in (w, None):
        exact, mag = _combine64(y, place, weights)
        bound = (k + 1) * 2.0 ** -23 * mag
        bound = bound + eps * (exact.abs() + bound)
        if out == "f16":
            bound = bound + 2.0 ** -25  # half a step of its subnormals
        for pad in (0, 3):
            full = torch.full((T + 2, H + pad), 9, device="cuda", dtype=TORCH[out])
            got = _ops().expert_combine(_padded(y, H + pad, float("nan")) if pad else y, place, weights, out_dtype=out,
                                        out=full[1:-1, :H])
            assert bool(((got.double() - exact).abs() <= bound).all())
            assert bool((got[T - 1] == 0).all())
            assert bool((full[0] == 9).all()) and bool((full[-1] == 9).all()) and bool((full[:, H:] == 9).all())


@gpu
@pytest.mark.parametrize("dtype,d", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (3, 2, 4, 3), (5, 3, 8, 8), (9, 8, 8, 33), (4, 9, 16, 40), (7, 5, 64, 2049),
                                     (65, 2, 8, 130), (2, 17, 32, 12), (3, 2, 4, 8191)])
def test_combine_grad(T, k, E, H, dtype, d):
    print(f"combine_grad {T}x{k} of {E}, {H} {dtype}, dout {d}", flush=True)
    _, src, place = _routing(T, k, E, T * 7 + H)
    y = torch.randn((T * k, H), device="cuda", generator=_gen(H)).to(TORCH[dtype])
    dout = torch.randn((T, H), device="cuda", generator=_gen(H + 1)).to(TORCH[d])
    w = torch.randn((T, k), device="cuda", generator=_gen(H + 2))
    n = int((src >= 0).sum())
    slot = src[:n].long()
    for weights in (w, None):
        want = torch.full((T * k, H), 9.0, dtype=TORCH[dtype], device="cuda")
        scale = w.flatten()[slot][:, None] if weights is not None else 1.0
        want[:n] = (scale * dout[slot // k].float()).to(TORCH[dtype])
        terms = y[:n].double() * dout[slot // k].double()
        exact = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(exact)
        exact[slot] = terms.sum(1)
        bound[slot] = (H + 1) * 2.0 ** -23 * terms.abs().sum(1)
        for pad in (0, 3):
            full = torch.full((T * k + 2, H + pad), 9.0, dtype=TORCH[dtype], device="cuda")
            dy, dw = _ops().expert_combine_grad(_padded(dout, H + pad, float("nan")) if pad else dout,
                                                _padded(y, H + 2 * pad, float("nan")) if pad else y, place, weights,
                                                dy=full[1:-1, :H])
            assert torch.equal(_bits(dy), _bits(want))
            assert bool(((dw.flatten().double() - exact).abs() <= bound).all())
            assert bool((full[0] == 9).all()) and bool((full[-1] == 9).all()) and bool((full[:, H:] == 9).all())


@gpu
def test_gradients_against_differences():
    """combine is linear in Y and in the weights: a step of any length gives the derivative.  Small whole
    numbers and weights of eighths, so that every sum is exact."""
    ops = _ops()
    T, k, E, H = 6, 3, 8, 20
    _, src, place = _routing(T, k, E, 5)
    g = _gen(9)
    y = torch.randint(-4, 5, (T * k, H), device="cuda", generator=g).float()
    w = torch.randint(-8, 9, (T, k), device="cuda", generator=g).float() / 8
    d = torch.randint(-4, 5, (T, H), device="cuda", generator=g).float()
    dy, dw = ops.expert_combine_grad(d, y, place, w, dy=torch.zeros_like(y))

    def loss(y, w):
        return float((ops.expert_combine(y, place, w).double() * d.double()).sum())

    base = loss(y, w)
    for r, c in ((0, 0), (3, 7), (11, 19), (T * k - 1, 4)):
        step = torch.zeros_like(y)
        step[r, c] = 1
        assert loss(y + step, w) - base == float(dy[r, c])
    for t in range(T):
        for j in range(k):
            step = torch.zeros_like(w)
            step[t, j] = 1
            assert loss(y, w + step) - base == float(dw[t, j])
    # dispatch's gradient is combine without weights
    x = torch.randint(-4, 5, (T, H), device="cuda", generator=g).float()
    rows = torch.randint(-4, 5, (T * k, H), device="cuda", generator=g).float()
    dx = ops.expert_combine(rows, place)

    def sent(x):
        return float((ops.expert_dispatch(x, place, out=torch.zeros_like(rows)).double() * rows.double()).sum())

    for t, c in ((0, 0), (3, 7), (5, 19)):
        step = torch.zeros_like(x)
        step[t, c] = 1
        assert sent(x + step) - sent(x) == float(dx[t, c])


@gpu
def test_infinities_and_nan_reach_only_their_tokens():
    ops = _ops()
    place = torch.tensor([[0, 2], [1, 3], [4, -1]], dtype=torch.int32, device="cuda")
    y = torch.ones((6, 64), dtype=torch.bfloat16, device="cuda")
    y[1, 3], y[2, 5], y[5] = float("inf"), float("nan"), float("nan")
    w = torch.tensor([[1.0, 0.5], [-1.0, 1.0], [2.0, float("inf")]], device="cuda")
    out = ops.expert_combine(y, place, w).float()
    assert torch.isnan(out[0, 5]) and out[1, 3] == float("-inf") and torch.isfinite(out).sum() == 3 * 64 - 2
    assert bool((out[2] == 2).all())


# ---- memory, streams, graphs ------------------------------------------------------------------------

@gpu
def test_rows_past_4_gib():
    """Y and the groups' rows past 2^32 bytes."""
    ops = _ops()
    R, H = 700000, 4096  # 5.7 GB of bf16
    y = torch.empty((R, H), dtype=torch.bfloat16, device="cuda")
    place = torch.tensor([[R - 1, 5], [600000, 300000]], dtype=torch.int32, device="cuda")
    x = torch.randint(-8, 9, (2, H), device="cuda").to(torch.bfloat16)
    ops.expert_dispatch(x, place, out=y)
    for t in range(2):
        for j in range(2):
            assert torch.equal(y[int(place[t, j])], x[t])
    w = torch.tensor([[1.0, 2.0], [0.5, -1.0]], device="cuda")
    assert torch.equal(ops.expert_combine(y, place, w), (x.float() * torch.tensor([[3.0], [-0.5]], device="cuda")).bfloat16())
    dw = ops.expert_combine_grad(x, y, place, w, dy=y.clone())[1]
    assert torch.equal(dw, (x.float() * x.float()).sum(1, keepdim=True).expand(2, 2))


@gpu
def test_wide_row_of_bytes_is_copied():
    x = torch.randint(0, 256, (1, (1 << 22) + 5), dtype=torch.uint8, device="cuda")
    place = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    out = _ops().expert_dispatch(x, place, out=torch.zeros((3, x.shape[1]), dtype=torch.uint8, device="cuda"))
    assert torch.equal(out[0], x[0]) and torch.equal(out[2], x[0]) and not bool(out[1].any())


@gpu
def test_on_another_stream():
    ops = _ops()
    s = torch.cuda.Stream()
    ids = torch.randint(0, 16, (500, 4), dtype=torch.int32, device="cuda")
    x = torch.randn((500, 128), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    off, src, place = ops.expert_sort(ids, 16, stream=s)
    rows = ops.expert_dispatch(x, place, stream=s)
    out = ops.expert_combine(rows, place, stream=s)
    s.synchronize()
    _check_sort(ids.cpu().numpy(), 16, (off, src, place))
    assert torch.equal(out, x + x + x + x)


@gpu
@pytest.mark.parametrize("T,k,E", [(8, 8, 64), (3000, 3, 40)])
def test_captured_layer_replays_with_other_choices(T, k, E):
    """Sort, dispatch and combine in one graph: each replay sorts the choices then in memory."""
    ops = _ops()
    H = 64
    ids = torch.zeros((T, k), dtype=torch.int32, device="cuda")
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((T, k), device="cuda")
    d = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    rows = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    need = tbg.expert_sort_workspace_query(T * k, E)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")

    def layer():
        off, src, place = ops.expert_sort(ids, E, workspace=ws if need else None)
        ops.expert_dispatch(x, place, out=rows)
        return (off, src, place, ops.expert_combine(rows, place, w), *ops.expert_combine_grad(d, rows, place, w, dy=dy))

    dy = torch.zeros_like(rows)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer()
    for step in range(4):
        g = _gen(step)
        ids.copy_(torch.randint(-1, E, (T, k), device="cuda", generator=g))
        x.copy_(torch.randn((T, H), device="cuda", generator=g))
        w.copy_(torch.randn((T, k), device="cuda", generator=g))
        d.copy_(torch.randn((T, H), device="cuda", generator=g))
        rows.zero_()
        dy.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        _check_sort(ids.cpu().numpy(), E, got[:3])
        rows.zero_()
        dy.zero_()
        want = layer()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), step


@gpu
def test_two_sorts_at_once():
    """Two streams, a workspace each."""
    ops = _ops()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ids = [torch.randint(0, 100, (60000,), dtype=torch.int32, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    got = [[ops.expert_sort(i, 100, stream=s) for i, s in zip(ids, streams)] for _ in range(4)]
    torch.cuda.synchronize()
    for round_ in got:
        for i, g in zip(ids, round_):
            _check_sort(i.cpu().numpy(), 100, g)


@gpu
def test_same_bits_every_time():
    ops = _ops()
    _, _, place = _routing(300, 6, 32, 3)
    y = torch.randn((1800, 1001), device="cuda", generator=_gen(1)).half()
    w, d = torch.randn((300, 6), device="cuda"), torch.randn((300, 1001), device="cuda").half()
    out = ops.expert_combine(y, place, w)
    dy, dw = ops.expert_combine_grad(d, y, place, w, dy=torch.zeros_like(y))
    for _ in range(3):
        assert torch.equal(out, ops.expert_combine(y, place, w))
        again = ops.expert_combine_grad(d, y, place, w, dy=torch.zeros_like(y))
        assert torch.equal(dy, again[0]) and torch.equal(dw, again[1])


@gpu
def test_helpers_refuse_on_the_device():
    ops = _ops()
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 8), device="cuda")
    w = torch.zeros((4, 2), device="cuda")
    calls = [
        lambda: ops.expert_sort(ids.long(), 4),
        lambda: ops.expert_sort(ids[:, :1], 4),
        lambda: ops.expert_dispatch(x[:3], ids),
        lambda: ops.expert_dispatch(x.double(), ids),
        lambda: ops.expert_dispatch(x, ids.flatten()),
        lambda: ops.expert_dispatch(x, ids, out=torch.zeros((8, 8), dtype=torch.float16, device="cuda")),
        lambda: ops.expert_dispatch(x, ids, out=torch.zeros((8, 7), device="cuda")),
        lambda: ops.expert_dispatch(x.t(), ids),
        lambda: ops.expert_combine(x, ids, w.double()),
        lambda: ops.expert_combine(x, ids, w[:3]),
        lambda: ops.expert_combine(x, ids, w, out_dtype="bf16"),
        lambda: ops.expert_combine(x, ids, w, out=x[:3]),
        lambda: ops.expert_combine(x.int(), ids, w),
        lambda: ops.expert_combine_grad(x.half(), x, ids, w),
        lambda: ops.expert_combine_grad(x[:3], x, ids, w),
        lambda: ops.expert_combine_grad(x, x, ids, w, dy=x.half()),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            print(i)


# ---- together ---------------------------------------------------------------------------------------

@gpu
def test_expert_layer_forward_and_backward():
    """A layer of experts as a training step runs it: sort, dispatch, two ragged products with a product in
    between, combine; and back.  Small whole numbers (weights of quarters): every sum and rounding is exact,
    so all of it equals the definition's gradients in 64 bits."""
    ops = _ops()
    T, k, E, H, F = 70, 2, 5, 24, 40
    g = _gen(3)
    ids = torch.argsort(torch.rand((T, E), device="cuda", generator=g), dim=1)[:, :k].to(torch.int32).contiguous()
    ids[T - 6:] = -1  # padded tokens

    def ints(shape, lo, hi):
        return torch.randint(lo, hi, shape, device="cuda", generator=g).float()

    x, w1, w2, dout = ints((T, H), -1, 2), ints((E, H, F), -1, 2), ints((E, F, H), -1, 2), ints((T, H), -1, 2)
    w = ints((T, k), -2, 3) / 2

    def half(t):
        return t.bfloat16()

    off, src, place = ops.expert_sort(ids, E)
    n = int(off[-1])
    rows = ops.expert_dispatch(half(x), place, out=torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda"))
    h = ops.gemm_grouped(rows, half(w1), off, out=torch.zeros((T * k, F), dtype=torch.bfloat16, device="cuda"))
    y = ops.gemm_grouped(h, half(w2), off, out_dtype="f32", out=torch.zeros((T * k, H), device="cuda"))
    out = ops.expert_combine(y, place, w)
    dy, dw = ops.expert_combine_grad(dout, y, place, w, dy=torch.zeros_like(y))
    dh = ops.gemm_grouped(half(dy), half(w2), off, b_layout="nk", out=torch.zeros_like(h))
    dw2 = ops.gemm_grouped_wgrad(h, half(dy), off)
    drows = ops.gemm_grouped(dh, half(w1), off, b_layout="nk", out_dtype="f32", out=torch.zeros((T * k, H), device="cuda"))
    dw1 = ops.gemm_grouped_wgrad(rows, dh, off)
    dx = ops.expert_combine(drows, place)
    # the definition, on the CPU in 64 bits
    leaves = [t.double().cpu().requires_grad_() for t in (x, w1, w2, w)]
    X, W1, W2, W = leaves
    want = torch.zeros((T, H), dtype=torch.float64)
    terms = []
    for t in range(T):
        total = torch.zeros(H, dtype=torch.float64)
        for j in range(k):
            e = int(ids[t, j])
            if e >= 0:
                total = total + W[t, j] * (X[t] @ W1[e] @ W2[e])
        terms.append(total)
    want = torch.stack(terms)
    (want * dout.double().cpu()).sum().backward()
    assert float(h[:n].float().abs().max()) <= 256 and float(dh[:n].float().abs().max()) <= 128  # whole in bf16
    assert torch.equal(out.double().cpu(), want.detach())
    for got, leaf in zip((dx, dw1, dw2, dw), leaves):
        assert torch.equal(got.double().cpu(), leaf.grad)


@gpu
def test_codes_are_dispatched():
    """Tokens quantised once to microscaled 4 bits; codes and scales go to the groups in place of the rows."""
    ops = _ops()
    T, k, E, K, N = 50, 2, 6, 256, 64
    g = _gen(8)
    x, b = torch.randn((T, K), device="cuda", generator=g), torch.randn((E, N, K), device="cuda", generator=g)
    off, src, place = _routing(T, k, E, 2)
    codes, scales = ops.mx4_quantize(x)
    c = ops.expert_dispatch(codes, place, out=torch.zeros((T * k, K // 2), dtype=torch.uint8, device="cuda"))
    s = torch.zeros((T * k, 16), dtype=torch.uint8, device="cuda")[:, :K // 32]
    ops.expert_dispatch(scales, place, out=s)
    rows = ops.expert_dispatch(x, place, out=torch.zeros((T * k, K), device="cuda"))
    c2, s2 = ops.mx4_quantize(rows)
    n = int(off[-1])
    assert torch.equal(c[:n], c2[:n]) and torch.equal(s[:n], s2[:n])
    bc, bs = ops.mx4_quantize(b)
    out = [ops.mx4_gemm_grouped(a, q, bc, bs, off, out=torch.zeros((T * k, N), dtype=torch.bfloat16, device="cuda"))
           for a, q in ((c, s), (c2, s2))]
    assert torch.equal(out[0], out[1])


# ---- rows past the cache, and batches of more than one launch -----------------------------------------

def _chunks(n, step=4096):
    return [slice(i, min(i + step, n)) for i in range(0, n, step)]


@gpu
@pytest.mark.parametrize("dtype,cols,pad", [(torch.uint8, 4099, 0), (torch.bfloat16, 2049, 5), (torch.float32, 1030, 0),
                                            (torch.float32, 1025, 3)])
@pytest.mark.parametrize("top_k", [3, 9])
def test_dispatch_of_rows_past_the_cache(dtype, cols, pad, top_k):
    """More than 256 MiB of the groups' rows: bit for bit, what lies around them as it was."""
    x1 = torch.empty(0, dtype=dtype)
    T = (256 << 20) // (cols * x1.element_size() * top_k) + 50
    print(f"dispatch {T}x{top_k}, {cols} {dtype}, past the cache", flush=True)
    _, src, place = _routing(T, top_k, 16, T + cols)
    n = int((src >= 0).sum())
    x = torch.randint(-100, 100, (T, cols), device="cuda", generator=_gen(cols)).to(dtype)
    out = torch.full((T * top_k + 2, cols + pad), 9, device="cuda", dtype=dtype)
    assert out[1:-1, :cols].numel() * out.element_size() >= 256 << 20
    _ops().expert_dispatch(_padded(x, cols + 2 * pad, 1) if pad else x, place, out=out[1:-1, :cols])
    for r in _chunks(n):
        assert torch.equal(_bits(out[1:-1, :cols][r]), _bits(x[(src[r] // top_k).long()]))
    assert bool((out[n + 1:] == 9).all()) and bool((out[0] == 9).all()) and bool((out[:, cols:] == 9).all())


@gpu
@pytest.mark.parametrize("dtype,out_dtype,cols,pad", [("bf16", "bf16", 2049, 5), ("bf16", "f32", 2048, 0), ("f16", "f16", 2050, 3),
                                                      ("f16", "f32", 2049, 1), ("f32", "f32", 1026, 1)])
@pytest.mark.parametrize("top_k", [5, 8, 10])
def test_combine_of_rows_past_the_cache(dtype, out_dtype, cols, pad, top_k):
    size = torch.empty(0, dtype=TORCH[dtype]).element_size()
    T = (256 << 20) // (cols * size * top_k) + 30
    print(f"combine {T}x{top_k}, {cols} {dtype} -> {out_dtype}, past the cache", flush=True)
    _, _, place = _routing(T, top_k, 16, T + cols)
    place[T - 1] = -1
    y = _padded(torch.randn((T * top_k, cols), device="cuda", generator=_gen(cols)).to(TORCH[dtype]), cols + pad, float("nan"))
    w = torch.randn((T, top_k), device="cuda", generator=_gen(cols + 1))
    full = torch.full((T + 2, cols + pad), 9, device="cuda", dtype=TORCH[out_dtype])
    eps = torch.finfo(TORCH[out_dtype]).eps / 2
    for weights in (w, None):
        got = _ops().expert_combine(y, place, weights, out_dtype=out_dtype, out=full[1:-1, :cols])
        for r in _chunks(T):
            exact, mag = _combine64(y, place[r], weights[r] if weights is not None else None)
            bound = (top_k + 1) * 2.0 ** -23 * mag
            bound = bound + eps * (exact.abs() + bound)
            if out_dtype == "f16":
                bound = bound + 2.0 ** -25  # half a step of its subnormals
            assert bool(((got[r].double() - exact).abs() <= bound).all())
        assert bool((got[T - 1] == 0).all())
        assert bool((full[0] == 9).all()) and bool((full[-1] == 9).all()) and bool((full[:, cols:] == 9).all())


@gpu
@pytest.mark.parametrize("dtype,d,cols,pad", [("bf16", "bf16", 2049, 5), ("bf16", "f32", 2048, 0), ("f16", "f16", 2050, 3),
                                              ("f16", "f32", 2049, 1), ("f32", "f32", 1026, 1)])
@pytest.mark.parametrize("top_k", [2, 4, 5, 9])
def test_combine_grad_of_rows_past_the_cache(dtype, d, cols, pad, top_k):
    """Y and dY of more than 256 MiB together: dY bit for bit, the weights' gradient within its sum's bound."""
    size = torch.empty(0, dtype=TORCH[dtype]).element_size()
    T = (128 << 20) // (cols * size * top_k) + 30
    print(f"combine_grad {T}x{top_k}, {cols} {dtype}, dout {d}, past the cache", flush=True)
    _, src, place = _routing(T, top_k, 16, T + cols)
    n = int((src >= 0).sum())
    y = _padded(torch.randn((T * top_k, cols), device="cuda", generator=_gen(cols)).to(TORCH[dtype]), cols + pad, float("nan"))
    dout = _padded(torch.randn((T, cols), device="cuda", generator=_gen(cols + 1)).to(TORCH[d]), cols + 2 * pad, float("nan"))
    w = torch.randn((T, top_k), device="cuda", generator=_gen(cols + 2))
    full = torch.full((T * top_k + 2, cols + pad), 9.0, dtype=TORCH[dtype], device="cuda")
    dy, dw = _ops().expert_combine_grad(dout, y, place, w, dy=full[1:-1, :cols])
    dw = dw.flatten()
    for r in _chunks(n):
        slot = src[r].long()
        rows = dout[slot // top_k].float()
        assert torch.equal(_bits(dy[r]), _bits((w.flatten()[slot][:, None] * rows).to(TORCH[dtype])))
        terms = y[r].double() * rows.double()
        assert bool(((dw[slot].double() - terms.sum(1)).abs() <= (cols + 1) * 2.0 ** -23 * terms.abs().sum(1)).all())
    assert bool((dw[place.flatten() < 0] == 0).all())
    assert bool((full[n + 1:] == 9).all()) and bool((full[0] == 9).all()) and bool((full[:, cols:] == 9).all())


@gpu
@pytest.mark.parametrize("top_k,cols", [(1, 3), (2, 9)])
def test_gradients_of_more_tokens_than_a_launch(top_k, cols):
    """A launch takes 2^22 - 1 tokens: those behind them have their own rows, weights and gradients."""
    T = (1 << 22) + 2
    print(f"combine_grad of {T} tokens", flush=True)
    g = _gen(cols)
    place = torch.randperm(T * top_k, device="cuda", generator=g).to(torch.int32).reshape(T, top_k)
    place[T - 3, 0] = place[7, 0] = -1
    y = torch.randint(-8, 9, (T * top_k, cols), device="cuda", generator=g).half()
    dout = torch.randint(-8, 9, (T, cols), device="cuda", generator=g).half()
    w = torch.randint(-8, 9, (T, top_k), device="cuda", generator=g).float()
    dy, dw = _ops().expert_combine_grad(dout, y, place, w, dy=torch.full_like(y, 99))
    # whole numbers: products up to 64 and sums up to 576, which fp16 and fp32 hold
    t, j = (place >= 0).nonzero(as_tuple=True)
    want = torch.full_like(y, 99)
    want[place[t, j].long()] = (w[t, j, None] * dout[t].float()).half()
    assert torch.equal(dy, want)
    held = place >= 0
    assert torch.equal(dw, (y[place.clamp(min=0).long()].float() * dout[:, None].float()).sum(-1) * held)


def _cut_rows(per_row):
    """Tokens of one launch, whose 16-byte or single-element units are counted in 32 bits, and some around the cut."""
    most = ((1 << 32) - 256) // per_row
    return most, most + 5, [0, 1, most - 2, most - 1, most, most + 1, most + 4]


@gpu
def test_dispatch_of_more_units_than_a_launch():
    most, T, at = _cut_rows(15)  # rows of 15 bytes go byte by byte
    print(f"dispatch of {T} tokens", flush=True)
    x = torch.zeros((T, 15), dtype=torch.uint8, device="cuda")
    place = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    for i, t in enumerate(at):
        x[t] = torch.arange(15, device="cuda") + 16 * i + 1
        place[t] = i + 1
    out = _ops().expert_dispatch(x, place, out=torch.full((len(at) + 2, 15), 250, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out[1:-1], x[torch.tensor(at, device="cuda")])
    assert bool((out[0] == 250).all()) and bool((out[-1] == 250).all())


@gpu
def test_combine_of_more_units_than_a_launch():
    most, T, at = _cut_rows(7)  # rows of 7 values go one by one
    print(f"combine of {T} tokens", flush=True)
    y = torch.randint(1, 9, (len(at), 7), device="cuda", generator=_gen(7)).bfloat16()
    place = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    w = torch.ones((T, 1), device="cuda")
    for i, t in enumerate(at):
        place[t] = i
        w[t] = i + 1
    out = torch.full((T, 7), 9, dtype=torch.bfloat16, device="cuda")
    _ops().expert_combine(y, place, w, out=out)
    for i, t in enumerate(at):
        assert torch.equal(out[t], (i + 1) * y[i])  # whole numbers up to 56
        out[t] = 0
    assert not any(bool(out[r].any()) for r in _chunks(T, 1 << 26))


@gpu
@pytest.mark.parametrize("dtype,cols", [(torch.uint8, 15), (torch.float16, 7), (torch.float32, 3)])
def test_dispatch_of_short_rows_past_the_cache(dtype, cols):
    """More than 256 MiB of rows below 16 bytes, which go element by element."""
    size, k = torch.empty(0, dtype=dtype).element_size(), 3
    T = (256 << 20) // (cols * size * k) + 3
    print(f"dispatch {T}x{k}, {cols} {dtype}, past the cache", flush=True)
    place = torch.randperm(T * k, device="cuda", generator=_gen(cols)).to(torch.int32).reshape(T, k)
    place[5, 1] = place[T - 1, 2] = -1
    x = torch.randint(0, 100, (T, cols), device="cuda", generator=_gen(cols + 1)).to(dtype)
    want = torch.full((T * k, cols), 101, device="cuda").to(dtype)
    t, j = (place >= 0).nonzero(as_tuple=True)
    want[place[t, j].long()] = x[t]
    got = _ops().expert_dispatch(x, place, out=torch.full((T * k, cols), 101, device="cuda").to(dtype))
    assert torch.equal(_bits(got), _bits(want))


@gpu
@pytest.mark.parametrize("dtype,out_dtype,cols", [("bf16", "bf16", 7), ("bf16", "f32", 5), ("f16", "f16", 7), ("f16", "f32", 3),
                                                  ("f32", "f32", 3)])
def test_combine_of_short_rows_past_the_cache(dtype, out_dtype, cols):
    """The same way back, in whole numbers: sums up to 5·8·8 are exact in every type but bf16, which rounds them once."""
    size, k = torch.empty(0, dtype=TORCH[dtype]).element_size(), 5
    T = (256 << 20) // (cols * size * k) + 3
    print(f"combine {T}x{k}, {cols} {dtype} -> {out_dtype}, past the cache", flush=True)
    place = torch.randperm(T * k, device="cuda", generator=_gen(cols)).to(torch.int32).reshape(T, k)
    place[5, 1] = place[T - 1, 2] = -1
    y = torch.randint(-8, 9, (T * k, cols), device="cuda", generator=_gen(cols + 1)).to(TORCH[dtype])
    w = torch.randint(-8, 9, (T, k), device="cuda", generator=_gen(cols + 2)).float()
    got = _ops().expert_combine(y, place, w, out_dtype=out_dtype)
    for r in _chunks(T, 1 << 20):
        terms = w[r][..., None] * (place[r] >= 0)[..., None] * y[place[r].clamp(min=0).long()].float()
        assert torch.equal(got[r], terms.sum(1).to(TORCH[out_dtype]))
