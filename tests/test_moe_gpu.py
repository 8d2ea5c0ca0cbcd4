"""Routing to experts and the combination of their rows against their definitions in 64
bits.  Experts, offsets, rows and slots are equal; a weight is rounded once from fp64."""
import numpy as np
import pytest
import torch

import moe_common as ref
import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _logits(tokens, experts, seed, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (1.5 * torch.randn(tokens, experts, generator=g)).to(dtype)


def _check(logits, top, **kw):
    """Routes of `logits` (on the GPU as given); kw as the call takes them, a bias in numpy."""
    l = logits.double().cpu().numpy()
    call = dict(kw)
    if kw.get("bias") is not None:
        call["bias"] = torch.from_numpy(kw["bias"].astype(np.float32)).cuda()
        kw["bias"] = call["bias"].double().cpu().numpy()
    r = rz.razer_moe_route(logits, top, **call)
    experts, weights = ref.route(l, top, **kw)
    assert np.array_equal(r.experts.cpu().numpy(), experts)
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(weights))
    # one rounding to fp32; the fp64 steps before it are off by some 2^-50
    ok = np.isnan(weights) | (np.abs(got - weights) <= np.abs(weights) * (2.0 ** -24 + 2.0 ** -44) + 2.0 ** -149)
    assert ok.all(), (got[~ok][:4], weights[~ok][:4])
    offsets, rows, slots = ref.order(experts, logits.shape[1])
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy(), slots)
    return r


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top", [(1, 1, 1), (1, 8, 2), (3, 7, 7), (1, 256, 8), (70, 64, 6), (5, 65, 3),
                                                (33, 128, 8), (4, 200, 32), (129, 257, 4), (2, 1000, 10), (9, 1024, 32),
                                                (500, 16, 1), (1025, 32, 4)])
def test_route(tokens, experts, top, score):
    for i, dtype in enumerate(DT.values()):
        _check(_logits(tokens, experts, tokens + experts + i, dtype).cuda(), top, score=score,
               renormalise=bool((tokens + i) & 1), scale=2.5 if i else 1.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top,groups,kept,best", [
    (40, 256, 8, 8, 4, 2), (40, 64, 6, 8, 3, 1), (7, 12, 2, 3, 1, 2), (9, 60, 5, 20, 7, 2), (5, 64, 3, 64, 9, 2),
    (6, 1024, 8, 16, 2, 2), (8, 320, 4, 5, 5, 1), (300, 16, 2, 2, 1, 2)])
def test_groups_and_bias(tokens, experts, top, groups, kept, best, score):
    rng = np.random.default_rng(tokens)
    for bias in (None, 0.2 * rng.normal(size=experts)):
        _check(_logits(tokens, experts, experts).cuda(), top, score=score, bias=bias, groups=groups, groups_kept=kept,
               group_best=best, renormalise=True, scale=2.5)


def test_ties_go_to_the_lowest():
    _check(torch.zeros(5, 100).cuda(), 7)
    _check(torch.zeros(5, 96).cuda(), 7, score="sigmoid", groups=8, groups_kept=3, group_best=2)
    l = _logits(200, 130, 1).mul(2).round().div(2)  # few different values
    for dtype in DT.values():
        _check(l.to(dtype).cuda(), 12)
        _check(l.to(dtype).cuda(), 12, score="sigmoid", groups=10, groups_kept=4, group_best=2, renormalise=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_bad_logits(score):
    inf, nan = float("inf"), float("nan")
    l = _logits(12, 70, 5)
    l[0] = -inf                       # padding
    l[1, 3:] = -inf                   # fewer experts than places
    l[2, ::2] = -inf
    l[3, 69], l[4, 0], l[5, 66] = nan, inf, -inf
    l[6], l[7] = 1e30, -1e30          # scores that are all equal, or all zero
    l[8], l[8, 40] = -200.0, 300.0
    l[9, :] = torch.finfo(torch.float32).min
    l[10, 64:] = -inf
    l[11, 7] = torch.finfo(torch.float32).max
    for renormalise in (False, True):
        _check(l.cuda(), 5, score=score, renormalise=renormalise)
        _check(l.cuda(), 5, score=score, groups=10, groups_kept=3, group_best=2, renormalise=renormalise)
        _check(l.cuda(), 1, score=score, groups=7, groups_kept=1, renormalise=renormalise)


def test_bias_that_masks():
    bias = np.zeros(32)
    bias[:20], bias[20], bias[25] = -np.inf, np.nan, np.inf
    for groups in (1, 4):
        _check(_logits(30, 32, 2).cuda(), 6, score="sigmoid", bias=bias, groups=groups, renormalise=True)
    _check(_logits(30, 32, 2).cuda(), 6, bias=np.full(32, -np.inf))
    _check(_logits(30, 32, 2).cuda(), 6, score="sigmoid", bias=-2 * np.ones(32), groups=4, groups_kept=2, group_best=2)


def test_strides_and_types():
    wide = _logits(50, 300, 3).cuda()
    for v in (wide[:, 5:69], wide[::3, :64], wide[:, :50].t(), wide[7:8, 3:20],
              wide[:1].expand(4, 300), wide[:, :1]):
        _check(v, min(3, v.shape[1]))


@pytest.mark.parametrize("tokens,experts,top", [(0, 8, 2), (300, 40, 5), (2500, 64, 6), (6000, 256, 8), (5000, 8, 2),
                                                (9001, 300, 3), (70000, 16, 2), (20000, 512, 8)])
def test_order(tokens, experts, top):
    """The order of many tokens' rows, from the experts that the call chose."""
    l = _logits(tokens, experts, tokens)
    if tokens > 10:
        l[torch.arange(0, tokens, 7)] = float("-inf")
        l[:, 0] += 4  # an expert that most tokens take
    r = rz.razer_moe_route(l.cuda(), top)
    chosen = r.experts.cpu().numpy().reshape(-1).astype(np.int64)
    flat = np.where(chosen < 0, experts, chosen)
    at = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[at], np.arange(experts + 1))
    n = tokens * top
    rows = np.where(np.arange(n) < offsets[experts], at // top, -1)
    slots = np.empty(n, dtype=int)
    slots[at] = np.arange(n)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.slots.cpu().numpy().reshape(-1), np.where(chosen < 0, -1, slots))
    bare = rz.razer_moe_route(l.cuda(), top, order=False)
    assert torch.equal(bare.experts, r.experts) and torch.equal(bare.weights, r.weights)
    assert bare.offsets is None and bare.rows is None and bare.slots is None


def test_given_results_and_workspace():
    l = _logits(77, 64, 9).cuda()
    want = rz.razer_moe_route(l, 6)
    out = rz.MoeRoutes(*(torch.full_like(t, 5) for t in want))
    ws = torch.empty(max(rz.razer_moe_workspace_bytes(77, 64, 6), 16), dtype=torch.uint8, device="cuda")
    for kw in (dict(out=out), dict(out=out, workspace=ws), dict(workspace=ws)):
        got = rz.razer_moe_route(l, 6, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        if "out" in kw:
            assert got is out


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("tokens,top,cols,add", [(1, 1, 8, False), (1, 8, 4096, True), (3, 2, 5, True), (7, 3, 1503, False),
                                                 (70, 6, 512, True), (300, 2, 2050, False), (2, 32, 20000, True)])
def test_combine(tokens, top, cols, add, dtype):
    """top + 1 fp32 additions, each off by at most 2^-24 of a partial sum, and the products by
    as much; the result is rounded once more."""
    rng = np.random.default_rng(tokens * top + cols)
    dt = DT[dtype]
    n = tokens * top + 3
    y = torch.from_numpy(rng.normal(size=(n, cols))).to(dt)
    slots = rng.permutation(n)[:tokens * top].reshape(tokens, top).astype(np.int32)
    slots[rng.random(slots.shape) < 0.1] = -1
    if slots.size > 4:
        slots.flat[3] = n
    weights = rng.random((tokens, top)).astype(np.float32)
    base = torch.from_numpy(3 * rng.normal(size=(tokens, cols))).to(dt) if add else None
    got = rz.razer_moe_combine(y.cuda(), torch.from_numpy(slots).cuda(), torch.from_numpy(weights).cuda(),
                               None if base is None else base.cuda())
    want, size = ref.combine(y.double().numpy(), slots, weights.astype(np.float64),
                             None if base is None else base.double().numpy())
    bound = (2 * top + 1) * 2.0 ** -24 * size + torch.finfo(dt).eps / 2 * np.abs(want) * 1.01
    bound += 2.0 ** -25 if dt is torch.float16 else 0  # half a step of its subnormals
    assert got.dtype is dt and (np.abs(got.double().cpu().numpy() - want) <= bound).all()


def test_combine_special():
    """Weights of NaN reach the result also through an empty slot; strides; out is add; nothing to do."""
    y = torch.randn(20, 64, device="cuda")
    slots = torch.tensor([[0, -1], [3, 4], [-1, -1]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, float("nan")], [0.5, 0.25], [0.0, 0.0]], device="cuda")
    out = rz.razer_moe_combine(y, slots, w)
    assert torch.isnan(out[0]).all() and (out[2] == 0).all()
    assert torch.equal(out[1], 0.5 * y[3] + 0.25 * y[4])
    h = torch.randn(3, 64, device="cuda")
    want = rz.razer_moe_combine(y, slots[1:], w[1:], h[1:])
    got = h.clone()
    assert rz.razer_moe_combine(y, slots[1:], w[1:], got[1:], out=got[1:]).data_ptr() == got[1:].data_ptr()
    assert torch.equal(got[1:], want) and torch.equal(got[0], h[0])
    wide = torch.zeros(20, 100, device="cuda")
    for at in (16, 3):
        wide[:, at:at + 64] = y
        assert torch.equal(rz.razer_moe_combine(wide[:, at:at + 64], slots[1:], w[1:], h[1:]), want)
    assert torch.equal(rz.razer_moe_combine(y.t().contiguous().t(), slots[1:], w[1:], h[1:]), want)
    assert rz.razer_moe_combine(y, slots[:0], w[:0]).shape == (0, 64)
    assert (rz.razer_moe_combine(y[:0], slots[2:], w[2:]) == 0).all()


def test_places_that_no_expert_takes_weigh_nothing():
    """... whatever the scale is, and whether or not there are scores to divide by."""
    logits = torch.full((3, 8), float("-inf"), device="cuda")
    logits[0, 5] = 1.0
    logits[1, 2] = -900.0  # a sigmoid that is 0 in 64 bits: a sum of nothing
    for scale in (float("inf"), -2.0):
        for renormalise in (False, True):
            for copies in (1, 7):
                r = rz.razer_moe_route(logits.repeat(copies, 1), 2, score="sigmoid", renormalise=renormalise, scale=scale)
                assert r.experts[:3].tolist() == [[5, -1], [2, -1], [-1, -1]]
                assert (r.weights[:, 1] == 0).all() and (r.weights[2::3] == 0).all()
    assert r.weights[1, 0] == 0 and r.weights[0, 0] == -2.0


@pytest.mark.parametrize("experts", [40, 100, 256, 257, 600])
@pytest.mark.parametrize("tokens", [7, 8, 9, 15, 16, 17, 31, 32, 33])
def test_where_one_workgroup_ends(tokens, experts):
    """Up to 32 tokens (16 of more than 64 experts, 8 of more than 256) are routed by one workgroup."""
    for top in (1, 32):
        logits = _logits(tokens, experts, tokens * experts).cuda()
        logits[tokens // 2] = float("-inf")
        logits[-1, 3] = float("nan")
        r = _check(logits, top, score="sigmoid")
        bare = rz.razer_moe_route(logits, top, score="sigmoid", order=False)
        assert torch.equal(bare.experts, r.experts) and bare.rows is None
        assert torch.equal(bare.weights.nan_to_num(-1.0), r.weights.nan_to_num(-1.0))


@pytest.mark.parametrize("dtype", sorted(DT))
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 24, 63, 100, 127, 129, 520, 2047, 2051, 4097])
def test_combine_widths(cols, dtype):
    """Rows shorter and longer than a workgroup's, that end inside 16 bytes, at every offset: nothing
    beside the result is written, nothing behind a row is read (it is NaN)."""
    dt, tokens, top = DT[dtype], 37, 3
    g = torch.Generator(device="cuda").manual_seed(cols)
    wide = torch.full((50, cols + 5), float("nan"), dtype=dt, device="cuda")
    buffer = torch.full((tokens * cols + 17,), 7.0, dtype=dt, device="cuda")
    slots = torch.randint(-1, 51, (tokens, top), generator=g, device="cuda").int()
    weights = torch.rand(tokens, top, generator=g, device="cuda")
    base = torch.randn(tokens, cols, generator=g, device="cuda").to(dt)
    for at in (0, 1, 4):
        y = wide[:, at:at + cols]
        wide.fill_(float("nan"))
        y.copy_(torch.randn(50, cols, generator=g, device="cuda"))
        out = buffer[at:at + tokens * cols].view(tokens, cols)
        buffer.fill_(7.0)
        rz.razer_moe_combine(y, slots, weights, base, out=out)
        want, size = ref.combine(y.double().cpu().numpy(), slots.cpu().numpy(), weights.double().cpu().numpy(),
                                 base.double().cpu().numpy())
        bound = (2 * top + 1) * 2.0 ** -24 * size + torch.finfo(dt).eps / 2 * np.abs(want) * 1.01
        bound += 2.0 ** -25 if dt is torch.float16 else 0  # half a step of its subnormals
        assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()
        assert (buffer[:at] == 7.0).all() and (buffer[at + tokens * cols:] == 7.0).all()
        place = base.clone()
        assert torch.equal(rz.razer_moe_combine(y, slots, weights, place, out=place), out)
