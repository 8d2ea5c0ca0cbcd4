"""Routing where a wave takes several tokens in turn, with groups and a bias, where the order
goes by sums of many blocks of many experts, and of as many tokens as a call takes; the
combination of a result that no launch has a thread for every element of.  Against the
definitions in 64 bits, whole tensors at a time."""
import numpy as np
import pytest
import torch

import nvfp4_razer_w4a16_amd as rz

pytestmark = pytest.mark.gpu
INF = np.inf


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def _ranks_below(key, count):
    """Which entries of each row are among its `count` largest, the lowest index first among equals."""
    first = np.argsort(-key, axis=-1, kind="stable")[..., :count]
    kept = np.zeros(key.shape, dtype=bool)
    np.put_along_axis(kept, first, True, -1)
    return kept


def _route(l, top, score, bias, groups, kept, best, renormalise, scale):
    """(experts, weights) of l [tokens, E], float64."""
    tokens, count = l.shape
    bad = np.isnan(l).any(1) | (l == INF).any(1)
    l = np.where(bad[:, None], 0.0, l)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == "sigmoid":
            s = 1.0 / (1.0 + np.exp(-l))
        else:
            s = np.exp(l - np.maximum(l.max(1, keepdims=True), -1e300))
            s = s / np.maximum(s.sum(1, keepdims=True), 1e-300)
    key = np.where(l == -INF, -INF, s if bias is None else s + bias)
    if groups > 1:
        parts = key.reshape(tokens, groups, -1)
        two = -np.sort(-parts, axis=-1)[..., :best]
        total = np.where(two[..., 0] == -INF, -INF, np.where(two == -INF, 0.0, two).sum(-1))
        stays = _ranks_below(total, kept) & (total > -INF)
        key = np.where(stays[..., None], parts, -INF).reshape(tokens, count)
    at = np.argsort(-key, axis=1, kind="stable")[:, :top]
    ok = np.take_along_axis(key, at, 1) > -INF
    w = np.where(ok, np.take_along_axis(s, at, 1), 0.0)
    if renormalise:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    experts = np.where(ok & ~bad[:, None], at, -1)
    return experts, np.where(bad[:, None], np.nan, w * scale)


def _order(experts, count):
    tokens, top = experts.shape
    flat = np.where(experts < 0, count, experts).reshape(-1)
    at = np.argsort(flat, kind="stable")
    offsets = np.searchsorted(flat[at], np.arange(count + 1))
    n = np.arange(flat.size)
    slots = np.empty(flat.size, dtype=int)
    slots[at] = n
    return offsets, np.where(n < offsets[count], at // top, -1), np.where(experts < 0, -1, slots.reshape(experts.shape))


# A wave takes two tokens where a block has 32, 17 or 9 of them to 16, 16 and eight waves (up to 128, 256
# and 512 experts), two to eight where it has 5 or 32 to four waves (above 512).  From 8193 tokens on there
# are more than 256 blocks.
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("tokens,experts,top,groups,kept,best", [
    (8200, 64, 6, 8, 3, 2), (8191, 128, 8, 8, 4, 1), (4200, 256, 8, 8, 4, 2), (8192, 256, 8, 8, 4, 2), (2100, 512, 8, 16, 4, 2),
    (1100, 1024, 16, 32, 8, 2), (9000, 1000, 10, 10, 4, 2), (20000, 600, 4, 1, 1, 1), (8200, 60, 3, 20, 5, 2)])
def test_many_tokens(tokens, experts, top, groups, kept, best, score):
    rng = np.random.default_rng(tokens + experts)
    l = (1.5 * rng.normal(size=(tokens, experts)) + 0.7 * rng.normal(size=experts)).astype(np.float32)
    l[5::97] = -INF                  # padding
    l[6::97, top - 1:] = -INF        # fewer experts than places, or as many, in one group
    l[7::97, ::2] = -INF
    l[8::197, experts - 1] = np.nan
    l[9::197, experts // 2] = INF
    l[10::41] = np.round(l[10::41])  # equal scores
    for i, dtype in enumerate((torch.float32, torch.bfloat16)):
        x = torch.from_numpy(l).to(dtype)
        bias = (0.1 * rng.normal(size=experts)).astype(np.float32)
        given = x.double().numpy()
        r = rz.razer_moe_route(x.cuda(), top, score=score, bias=torch.from_numpy(bias).cuda(), groups=groups,
                               groups_kept=kept, group_best=best, renormalise=not i, scale=2.5)
        want, weights = _route(given, top, score, bias.astype(np.float64), groups, kept, best, not i, 2.5)
        assert np.array_equal(r.experts.cpu().numpy(), want)
        got = r.weights.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(weights))
        # one rounding to fp32; the fp64 steps before it are off by some 2^-50
        ok = np.isnan(weights) | (np.abs(got - weights) <= np.abs(weights) * (2.0 ** -24 + 2.0 ** -44) + 2.0 ** -149)
        assert ok.all(), (got[~ok][:4], weights[~ok][:4])
        for g, w in zip((r.offsets, r.rows, r.slots), _order(want, experts)):
            assert np.array_equal(g.cpu().numpy(), w)


@pytest.mark.parametrize("tokens,experts,top", [((1 << 20) + 7, 8, 2), ((1 << 22) + 1, 16, 16), (1 << 26, 2, 1)])
def test_without_an_order(tokens, experts, top):
    """Up to 2^26 tokens, of which no order is made above 2^20."""
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    l = torch.randn(tokens, experts, generator=gen, device="cuda")
    l[::1001] = float("-inf")
    r = rz.razer_moe_route(l, top, order=False)
    assert r.offsets is None and r.rows is None and r.slots is None
    best, at = torch.sort(l, dim=1, descending=True, stable=True)
    at = torch.where(best > float("-inf"), at, -1)[:, :top]
    assert torch.equal(r.experts.long(), at)
    for a in range(0, tokens, 1 << 22):
        s = slice(a, a + (1 << 22))
        p = torch.softmax(l[s].double(), 1).gather(1, at[s].clamp_min(0))
        p = torch.where(at[s] < 0, 0.0, p)
        assert ((r.weights[s].double() - p).abs() <= p * (2.0 ** -24 + 2.0 ** -44)).all()


def test_combine_into_more_than_a_launch_has_threads():
    """2^34 - 2^18 results in fp32, four to a thread."""
    tokens, cols = 65535, 1 << 18
    y = torch.randn(2, cols, device="cuda")
    slots = (torch.arange(tokens, device="cuda", dtype=torch.int32) % 3 - 1)[:, None].contiguous()
    weights = (torch.arange(tokens, device="cuda") % 5 + 1.0)[:, None]
    out = torch.full((tokens, cols), 7.0, device="cuda")
    rz.razer_moe_combine(y, slots, weights, out=out)
    for a in range(0, tokens, 4096):
        s = slots[a:a + 4096, 0].long()
        want = torch.where(s[:, None] < 0, 0.0, y[s.clamp_min(0)]) * weights[a:a + 4096]
        assert torch.equal(out[a:a + 4096], want)
