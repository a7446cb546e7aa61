"""How far the attention's weights are kept (``spec_verify_attend``): rows in which a few positions tower above all others, as
a model's first tokens do, levels that change along a context, weights of every size, scales that are no numbers.

Everything is compared with 64 bits.  The bound of an output entry is that of weights of eight significant bits, plus 2^-31 of
the row's largest weight for each position."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.test_gpu_step_operators import attend_case, gen, sv  # noqa: F401  (sv is a fixture)

pytestmark = pytest.mark.gpu
i32, f32, bf16, f8, f64 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn, torch.float64


def flat_case(B, heads, group, dim, context, nodes, tokens=64, seed=1):
    """Chains of `nodes` after `context` positions in a cache of zeros with scales of 1 whose pages lie in order: K and V as
    [B, heads, positions, dim] views of it."""
    n = context + 1 + nodes
    cols = (n + tokens - 1) // tokens
    pages = B * cols
    raw = [torch.zeros(pages, heads, tokens, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones(pages, heads, 1, device="cuda") for _ in range(2)]
    table = torch.arange(pages, dtype=i32, device="cuda").view(B, cols)
    q = torch.zeros(B * (nodes + 1), heads * group, dim, dtype=bf16, device="cuda")
    return dict(q=q, cache=[t.view(f8) for t in raw] + scales, page_table=table,
                context=torch.full((B,), context, dtype=i32, device="cuda"),
                node_start=torch.arange(B + 1, device="cuda").to(i32) * nodes), n


def put(c, which, x):
    """x [B, heads, positions, dim] becomes the entries of k or v (scales are left)."""
    t = c["cache"][which]
    B, cols = c["page_table"].shape
    heads, tokens, dim = t.shape[1:]
    full = torch.zeros(B, heads, cols * tokens, dim, device="cuda")
    full[:, :, :x.shape[2]] = x
    e = full.view(B, heads, cols, tokens, dim).transpose(1, 2).reshape(-1, heads, tokens, dim)
    t.view(torch.uint8).copy_(e.to(f8).view(torch.uint8))


def take(c, which, n):
    """The first n positions as values: [B, heads, n, dim] in 64 bits."""
    t, s = c["cache"][which].to(f32).to(f64), c["cache"][2 + which].to(f64)
    x = t * s.repeat_interleave(t.shape[2] // s.shape[2], 2)[..., None]
    B, cols = c["page_table"].shape
    x = x.view(B, cols, *x.shape[1:]).transpose(1, 2)
    return x.reshape(B, x.shape[1], -1, x.shape[-1])[:, :, :n]


def assert_weights(got, c, n, what=""):
    """Chains.  A logit is off by d: the tensor core's sums of 2 dim products in steps of 32, which cut off less than 2^-23 of
    the magnitudes for each and for the sum; three fp32 products with scales and the difference to the reference (2^-24 of
    the largest magnitude each); a query entry may be off by 2^-17.8 of its row's largest.  Weights are rounded to eight bits, 2^-8, or by
    2^-31 of the largest; products with V are summed like those with K, over n / 32 steps and a few joins; the sum of the
    weights is off by 2^-24 an addition; the result is rounded to bf16."""
    B = c["context"].shape[0]
    rows = c["q"].shape[0] // B
    dim = c["q"].shape[2]
    k, v = take(c, 0, n), take(c, 1, n)
    heads = k.shape[1]
    q = c["q"].to(f64).view(B, rows, heads, -1, dim)
    scale = dim ** -0.5
    s = scale * torch.einsum("brhgd,bhnd->bhgrn", q, k)
    mag = scale * torch.einsum("brhgd,bhnd->bhgrn", q.abs(), k.abs())
    first = n - rows
    hidden = torch.arange(n, device="cuda")[None, :] > first + torch.arange(rows, device="cuda")[:, None]
    s = s.masked_fill(hidden, -float("inf"))
    d = mag * (8 * (dim / 16 + 1) + 8) * 2.0 ** -23 + 5 * 2.0 ** -24 * s.masked_fill(hidden, 0).abs().amax(-1, keepdim=True)
    most = q.abs().amax(-1).permute(0, 2, 3, 1)
    d = d + scale * k.abs().sum(-1)[:, :, None, None] * most[..., None] * 2.0 ** -17.8
    p = torch.softmax(s, -1)
    o = torch.einsum("bhgrn,bhnd->bhgrd", p, v)
    size = c["cache"][3].to(f64)
    assert float(size.min()) == float(size.max()) == 1.0
    level = p.amax(-1, keepdim=True)
    weight = p * (2.0 * d + 2.0 ** -8 + (n / 16 + 8) * 33 * 2.0 ** -23) + (p > 0) * level * 2.0 ** -31
    err = torch.einsum("bhgrn,bhnd->bhgrd", weight, v.abs()) + ((p * 2 * d).sum(-1, keepdim=True) + n * 2.0 ** -24) * o.abs()
    bound = err * 1.01 + (o.abs() + err) * 2.0 ** -8
    have = got.to(f64).view(B, rows, heads, -1, dim).permute(0, 2, 3, 1, 4)
    far = (have - o).abs()
    assert bool((far <= bound).all()), (what, float((far / bound).max()), float((far / o.abs().clamp_min(1e-300)).max()))


def towering_case(B, heads, group, dim, context, nodes, at, gap, spread, seed=3):
    """Positions `at` stand about `gap` above the others' logits, whose standard deviation is `spread`, and have values of 0;
    the others' values are positive."""
    g = gen(seed)
    c, n = flat_case(B, heads, group, dim, context, nodes)
    k = torch.randn(B, heads, n, dim, generator=g, device="cuda") * (spread > 0)
    k[..., 0] = 0
    v = 0.5 + torch.rand(B, heads, n, dim, generator=g, device="cuda")
    for j, (p, high) in enumerate(zip(at, gap)):
        k[:, :, p] = 0
        k[:, :, p, 0] = high * dim ** 0.5 / 8
        v[:, :, p] = 0
    put(c, 0, k), put(c, 1, v)
    c["q"].copy_(torch.randn(c["q"].shape, generator=g, device="cuda") * spread)
    c["q"][..., 0] = 8
    return c, n


@pytest.mark.parametrize("gap", [8.0, 9.5, 10.3, 10.5, 11.0, 12.0, 13.0, 16.0, 30.0])
@pytest.mark.parametrize("spread", [0.0, 0.5, 1.2])
@pytest.mark.parametrize("B,heads,group,dim,context,nodes", [
    (40, 8, 1, 64, 1999, 0), (40, 4, 4, 128, 2000, 3), (40, 4, 8, 64, 2100, 4), (300, 1, 4, 128, 99, 0), (1, 1, 4, 128, 30000, 1)])
def test_attend_a_first_position_above_all_others(sv, gap, spread, B, heads, group, dim, context, nodes):
    # units that are whole for the most part (one block of columns, two of them), short contexts, one that is cut
    c, n = towering_case(B, heads, group, dim, context, nodes, [0], [gap], spread)
    assert_weights(sv.attend_tree(**c), c, n)


@pytest.mark.parametrize("gap", [9.0, 12.0, 15.0])
@pytest.mark.parametrize("spread", [0.0, 0.5])
@pytest.mark.parametrize("group,dim,nodes", [(2, 64, 0), (4, 128, 4), (8, 64, 4)])
def test_attend_four_first_positions_of_different_heights(sv, gap, spread, group, dim, nodes):
    c, n = towering_case(20, 8, group, dim, 1500, nodes, [0, 1, 2, 3], [gap, gap - 1.5, gap - 4, gap - 2.2], spread)
    assert_weights(sv.attend_tree(**c), c, n)


@pytest.mark.parametrize("gap", [9.0, 11.0, 14.0])
@pytest.mark.parametrize("every", [100, 128, 1000])
@pytest.mark.parametrize("group,dim,nodes", [(4, 128, 0), (8, 64, 4)])
def test_attend_positions_above_the_others_again_and_again(sv, gap, every, group, dim, nodes):
    at = list(range(5, 4000, every))
    c, n = towering_case(20, 8, group, dim, 4000, nodes, at, [gap + (i * 7 % 5) * 0.4 for i in range(len(at))], 0.5)
    assert_weights(sv.attend_tree(**c), c, n)


@pytest.mark.parametrize("rise", [-40.0, -20.0, -12.0, 12.0, 40.0])
@pytest.mark.parametrize("group,dim", [(2, 128), (12, 64)])
def test_attend_levels_that_change_along_a_context(sv, rise, group, dim):
    # logits that rise or fall evenly, by `rise` over the whole context, and a step of 14 in the middle
    c, n = flat_case(30, 8, group, dim, 2500, 3)
    g = gen(5)
    k = torch.randn(30, 8, n, dim, generator=g, device="cuda") * 0.5
    ramp = torch.linspace(0, rise, n, device="cuda") + 14.0 * (torch.arange(n, device="cuda") > 1300)
    k[..., 0] = ramp * dim ** 0.5 / 8
    k[..., 0].clamp_(-440, 440)
    put(c, 0, k), put(c, 1, 0.5 + torch.rand(k.shape, generator=g, device="cuda"))
    c["q"].copy_(torch.randn(c["q"].shape, generator=g, device="cuda"))
    c["q"][..., 0] = 8
    assert_weights(sv.attend_tree(**c), c, n)


def test_attend_spread_logits(sv):
    # from nearly equal ones to those of which a few take everything, row by row
    c, n = flat_case(12, 8, 8, 128, 1700, 4)
    g = gen(6)
    put(c, 0, torch.randn(12, 8, n, 128, generator=g, device="cuda"))
    put(c, 1, torch.randn(12, 8, n, 128, generator=g, device="cuda"))
    spread = torch.linspace(0.1, 8, 64, device="cuda")[:, None]
    c["q"].copy_(torch.randn(c["q"].shape, generator=g, device="cuda") * spread)
    assert_weights(sv.attend_tree(**c), c, n)


def test_attend_weights_of_every_size_above_the_reference(sv):
    # The third tile, the second one of its group, has one position by 0 to 12 bits above the first one's largest: nearly all
    # of the weight, so that its rounding is that of the result.  64 heights of 64 query heads.
    c, n = flat_case(1, 1, 64, 64, 400, 0)
    k = torch.zeros(1, 1, n, 64, device="cuda")
    k[0, 0, :, 0] = -20.0
    k[0, 0, 3, 0], k[0, 0, 3, 1] = 0.0, 0.0
    k[0, 0, 300, 0], k[0, 0, 300, 1] = 0.0, 1.0
    v = torch.zeros_like(k)
    v[0, 0, 300] = 1.0
    put(c, 0, k), put(c, 1, v)
    c["q"][..., 0] = 8.0 * 8.0 ** 0.5
    # bf16 queries, exact as they are compared
    c["q"][0, :, 1] = (torch.arange(64, device="cuda") / 64 * 12 * np.log(2.0) * 8).to(bf16)
    got = sv.attend_tree(**c).to(f64)[0, :, 0]
    q1 = c["q"][0, :, 1].to(f64)
    want = torch.softmax(torch.stack([torch.zeros_like(q1), q1 / 8.0]), 0)[1]
    # 2^-8 for the weight, 2^-16 for all else, half a bf16 step
    half = torch.exp2(torch.floor(torch.log2(got)) - 8)
    assert bool(((got - want).abs() <= want * (2.0 ** -8 + 2.0 ** -16) + half).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", [2, 3])
def test_attend_scales_that_are_no_numbers_reach_the_rows_that_see_them(sv, bad, which):
    context, sizes = [100, 127, 60], [7, 3, 0]
    c = attend_case(21, context, sizes, 2, 2, 64, 16, 1)
    want = sv.attend_tree(**c).clone()
    table = c["page_table"].tolist()
    for b, (n, m) in enumerate(zip(context, sizes)):  # behind the last row: nobody
        for p in range(n + 1 + m, 16 * len(table[b])):
            c["cache"][which][table[b][p // 16], :, p % 16] = bad
    assert torch.equal(sv.attend_tree(**c), want)
    p = context[0] + 1 + 2  # node 2, key head 1
    c["cache"][which][table[0][p // 16], 1, p % 16] = bad
    got = sv.attend_tree(**c)
    parent = c["parent"].tolist()
    lost = [i for i in range(8) if 2 in ref.path_of(parent, i)]
    assert 3 in lost and len(lost) < 7
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    keep[lost, 2:4] = False
    assert torch.equal(got[keep], want[keep])
    if bad != bad or which == 3:
        assert bool(torch.isnan(got[~keep]).all())


def test_attend_a_nan_far_below_the_others_is_not_lost(sv):
    # Two tiles at the end whose logits lie 100 below all others': the last one's only positions have a page that is none.
    # However the tiles are cut, the row becomes NaN.
    for n in range(20, 320, 7):
        c, total = flat_case(1, 1, 1, 64, 128 * n + 10, 0, tokens=128)
        k = torch.zeros(1, 1, total, 64, device="cuda")
        k[:, :, 128 * (n - 1):, 0] = -100.0
        put(c, 0, k)
        c["q"][..., 0] = 8.0
        assert not bool(torch.isnan(sv.attend_tree(**c)).any())
        c["page_table"][0, n] = -1
        assert bool(torch.isnan(sv.attend_tree(**c)).all()), n


def test_attend_scales_too_far_apart_are_told(sv):
    # The first tile's values have the least scale that there is.  Others 2^110 times as large are added as they should be, and
    # 2^125 times as large make a row NaN, or, where its units are cut behind that tile, are added as they should be too.
    c, n = flat_case(40, 8, 4, 64, 700, 1)
    g = gen(9)
    put(c, 0, torch.randn(40, 8, n, 64, generator=g, device="cuda"))
    put(c, 1, 1.0 + torch.rand(40, 8, n, 64, generator=g, device="cuda"))
    c["q"].copy_(torch.randn(c["q"].shape, generator=g, device="cuda"))
    first, others = c["page_table"][:, :2].long(), c["page_table"][:, 2:].long()
    c["cache"][3][first] = 0.0
    want = sv.attend_tree(**c).float()
    c["cache"][3][first] = 2.0 ** -100
    for power in (10, 25):
        c["cache"][3][others] = 2.0 ** power
        got = sv.attend_tree(**c).float() * 2.0 ** -power
        none = torch.isnan(got)
        assert bool((none.any(-1) == none.all(-1)).all()) and bool(none.any()) == (power == 25)
        # two results of the same weights, each rounded to bf16, and fp16 weights
        assert bool((((got - want).abs() <= want.abs() * (2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10)) | none).all())
