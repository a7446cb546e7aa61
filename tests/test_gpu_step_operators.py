"""The operators around a tree's target pass on the GPU: penalties on logits rows, the 8-bit cache in pages, the attention
over it, and a run of them together, against 64-bit implementations.  Bounds are derived beside them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import operators_reference as op_ref
from tests import step_reference as ref

pytestmark = pytest.mark.gpu
i32, f32, bf16, f8 = torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_online_gb300 as pkg
    from speculative_decoding_verification_online_gb300 import build as B
    B.build()
    pkg.load()
    return pkg


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ints(*v):
    return torch.tensor(v, dtype=i32, device="cuda")


def random_trees(seed, sizes):
    """node_start and parents of trees of the given numbers of nodes."""
    r = np.random.RandomState(seed)
    parent = [int(r.randint(max(-1, i - 6), i)) for n in sizes for i in range(n)]
    return ints(0, *np.cumsum(sizes).tolist()), torch.tensor(parent, dtype=i32, device="cuda")


# ------------------------------------------------------------- penalties

def penalty_case(seed, V, sizes, cap, dtype=f32, words=True, pad=0, offset=0, chain=False):
    g = gen(seed)
    node_start, parent = random_trees(seed, sizes)
    B, total = len(sizes), int(sum(sizes))
    rows = total + B
    store = torch.full((offset + rows * (V + pad),), float("nan"), dtype=dtype, device="cuda")
    logits = store[offset:].view(rows, V + pad)[:, :V]
    logits.copy_(torch.randn(rows, V, generator=g, device="cuda") * 3)
    few = max(1, min(V, 40))

    def toks(*shape):
        t = torch.randint(0, few, shape, generator=g, device="cuda")
        return ((t * 7919) % V).to(i32)

    c = dict(logits=logits, history=toks(B, cap + 3)[:, 1:cap + 1], tokens=toks(total), parent=None if chain else parent,
             node_start=node_start, history_len=torch.randint(0, cap + 1, (B,), generator=g, device="cuda").to(i32))
    c["history_len"][-1] = cap
    c["prompt_len"] = (c["history_len"] // 3).to(i32)
    c["repetition"] = 1.0 + torch.rand(B, generator=g, device="cuda")
    c["frequency"] = torch.rand(B, generator=g, device="cuda") - 0.3
    c["presence"] = torch.rand(B, generator=g, device="cuda") - 0.3
    n = 5 * B
    c["bias"] = (torch.arange(0, n + 1, 5, device="cuda").to(i32), toks(n), torch.randn(n, generator=g, device="cuda") * 3)
    if words:
        c["mask"] = torch.randint(-2 ** 31, 2 ** 31, (rows, (V + 31) // 32 + 1), generator=g, device="cuda").to(i32)
        c["mask"][::2, ::2] = -1
        c["mask"][1::3, 1::2] = 0
        c["mask_row"] = torch.arange(rows, device="cuda").flip(0).to(i32)
        c["mask_row"][::4] = -1
    return c


def assert_penalties(got, c, what=""):
    """At most ten roundings of fp32 to values no larger than twice the sum of the magnitudes, then one to the type."""
    want, size = ref.penalties(**c)
    have = ref.doubles(got)
    assert np.array_equal(np.isnan(have), np.isnan(want)), what
    inf = np.isinf(want)
    assert np.array_equal(have[inf], want[inf]), what
    fine = np.isfinite(want)
    bound = 20 * 2.0 ** -24 * (size + np.abs(np.where(fine, want, 0.0)))
    if got.dtype == bf16:
        bound = bound + (np.abs(np.where(fine, want, 0.0)) + bound) * 2.0 ** -8
    assert np.all(np.abs(have[fine] - want[fine]) <= bound[fine]), what


@pytest.mark.parametrize("V,sizes,cap", [
    (1, [0], 0), (7, [1, 0, 3], 5), (31, [4], 9), (32, [2, 2], 40), (33, [0, 0], 1), (1000, [5], 33), (1024, [0, 21, 7], 200),
    (1025, [3], 64), (5000, [1] * 9, 17), (32000, [4], 300), (8191, [30, 2], 1000), (70001, [2, 0, 1], 4097)])
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("out", ["same", "new", "f32"])
def test_penalties_sizes(sv, V, sizes, cap, dtype, out):
    c = penalty_case(V + cap, V, sizes, cap, dtype)
    before = c["logits"].clone()
    o = c["logits"] if out == "same" else None if out == "new" else torch.full(before.shape, 3.0, device="cuda")
    args = [c[k] for k in ("logits", "history", "history_len", "tokens", "parent", "node_start")]
    kw = {k: c[k] for k in ("prompt_len", "repetition", "frequency", "presence", "bias", "mask", "mask_row")}
    got = sv.penalize(*args, **kw, out=o)
    assert got.dtype == (f32 if out == "f32" else dtype)
    assert_penalties(got, dict(c, logits=before))
    if out != "same":
        assert torch.equal(c["logits"], before)


@pytest.mark.parametrize("leave", ["prompt_len", "repetition", "frequency", "presence", "bias", "mask", "parent", "all"])
@pytest.mark.parametrize("place", ["same", "new"])
def test_penalties_each_may_be_left_out(sv, leave, place):
    c = penalty_case(11, 3000, [6, 0, 12], 50, bf16)
    gone = ("prompt_len", "repetition", "frequency", "presence", "bias", "mask", "mask_row") if leave == "all" else (
        ("mask", "mask_row") if leave == "mask" else (leave,))
    for k in gone:
        c[k] = None
    before = c["logits"].clone()
    got = sv.penalize(**c, out=c["logits"] if place == "same" else None)
    assert_penalties(got, dict(c, logits=before))


@pytest.mark.parametrize("pad,offset", [(1, 0), (8, 0), (3, 1), (0, 8), (4, 4)])
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("place", ["same", "new"])
def test_penalties_strides_and_alignment(sv, pad, offset, dtype, place):
    c = penalty_case(5 + pad, 2051, [3, 9], 77, dtype, pad=pad, offset=offset)
    before = c["logits"].clone()
    rows, V = before.shape
    store = torch.full((rows, V + 5), 7.0, dtype=dtype, device="cuda")
    got = sv.penalize(**c, out=c["logits"] if place == "same" else store[:, 2:V + 2])
    assert_penalties(got, dict(c, logits=before))
    if place == "new":
        assert bool((store[:, :2] == 7).all()) and bool((store[:, V + 2:] == 7).all())


def test_penalties_masked_places_may_hold_anything_and_rows_may_be_left_empty(sv):
    c = penalty_case(3, 1500, [2, 2], 30)
    c["mask"][:] = 0
    c["mask"][:, 5] = 8
    c["mask_row"] = None
    c["logits"][0, :160] = float("nan")
    c["logits"][1, :160] = float("inf")
    c["logits"][2, :160] = -3.3895313892515355e+38
    c["mask"][3] = 0  # nothing is allowed
    before = c["logits"].clone()
    got = sv.penalize(**c)
    assert_penalties(got, dict(c, logits=before))
    assert bool((got[3] == float("-inf")).all())
    assert bool(torch.isnan(sv.softmax(got, 1.0)[3]).all())
    # places that are not masked keep what they hold
    c["mask"] = None
    got = sv.penalize(**c, out=c["logits"])
    assert_penalties(got, dict(c, logits=before))


def test_penalties_of_padded_and_invalid_sequences(sv):
    V, sizes = 1200, [2, 3, 1, 2, 2, 4, 3, 2]
    c = penalty_case(8, V, sizes, 20)
    starts = [0, *np.cumsum(sizes).tolist()]
    c["history_len"][0] = -1  # padded
    c["repetition"][1] = 0.0
    c["frequency"][2] = float("nan")
    c["history_len"][3] = 21
    c["bias"][0][5] = c["bias"][0][4] - 1  # sequence 4 has a range that falls
    c["parent"][starts[5] + 2] = 2  # its own parent: rows behind it are lost
    c["parent"][starts[5] + 3] = 2
    c["mask_row"][starts[6] + 6 + 1] = len(c["mask"])
    c["presence"][7] = float("inf")
    out = torch.full(c["logits"].shape, 5.0, device="cuda")
    got = sv.penalize(**c, out=out)
    rows = lambda b: slice(starts[b] + b, starts[b + 1] + b + 1)  # noqa: E731
    assert bool((got[rows(0)] == 5).all())
    for b in (1, 2, 3, 4, 7):
        assert bool(torch.isnan(got[rows(b)]).all()), b
    five, six = got[rows(5)], got[rows(6)]
    assert bool(torch.isnan(five[3:]).all()) and not bool(torch.isnan(five[:3]).any())
    assert bool(torch.isnan(six[1]).all()) and not bool(torch.isnan(six[[0, 2, 3]]).any())
    # a range of nodes that is none: its rows are not known, and nothing is written
    c = penalty_case(9, V, [2, 2, 2], 20)
    c["node_start"][1] = 70
    out = torch.full(c["logits"].shape, 5.0, device="cuda")
    got = sv.penalize(**c, out=out)
    assert bool((got[:6] == 5).all())


def test_penalties_tokens_outside_count_nothing(sv):
    c = penalty_case(2, 100, [3], 12)
    c["history"][0, 3:6] = ints(-1, 100, 2 ** 31 - 1)
    c["tokens"][1] = -5
    c["bias"][1][2] = 100
    before = c["logits"].clone()
    got = sv.penalize(**c, out=c["logits"])
    c["bias"] = (ints(0, 4), c["bias"][1][[0, 1, 3, 4]], c["bias"][2][[0, 1, 3, 4]])
    assert_penalties(got, dict(c, logits=before))


def test_penalties_the_deepest_chain_and_one_token_everywhere(sv):
    n, V = 256, 5000
    c = penalty_case(4, V, [n, 0], 100, chain=True)
    c["tokens"][:] = 4999
    c["tokens"][::2] = 17
    c["history"][:] = 17
    c["mask"] = c["mask_row"] = None
    before = c["logits"].clone()
    assert_penalties(sv.penalize(**c, out=c["logits"]), dict(c, logits=before))


def test_penalties_rows_past_2_to_31_entries(sv):
    V, rows = 1 << 22, 520
    logits = torch.zeros(rows, V, dtype=bf16, device="cuda")
    sizes = [0] * rows
    node_start = torch.zeros(rows + 1, dtype=i32, device="cuda")
    tokens = torch.empty(0, dtype=i32, device="cuda")
    history = torch.full((rows, 1), V - 1, dtype=i32, device="cuda")
    got = sv.penalize(logits, history, torch.ones(rows, dtype=i32, device="cuda"), tokens, None, node_start,
                      presence=torch.arange(rows, device="cuda") % 7 + 1.0, out=logits)
    want = -(torch.arange(rows, device="cuda") % 7 + 1.0)
    assert torch.equal(got[:, -1].float(), want) and int((got != 0).sum()) == len(sizes)


# ------------------------------------------------------------- the cache

def make_cache(seed, pages, heads, tokens, dim, block, layers=None, order="head"):
    g = gen(seed)
    lead = () if layers is None else (layers,)

    def entries():
        shape = (heads, tokens) if order == "head" else (tokens, heads)
        x = torch.randint(0, 256, lead + (pages, *shape, dim), generator=g, device="cuda").to(torch.uint8)
        x = torch.where((x & 0x7f) == 0x7f, x - 1, x)  # no NaN
        x = x.view(f8)
        return x if order == "head" else x.transpose(-2, -3)

    def scales():
        return torch.exp(torch.randn(*lead, pages, heads, tokens // block, generator=g, device="cuda") * 0.7 - 5.0)

    return [entries(), entries(), scales(), scales()]


def make_table(seed, lengths, tokens, spare=3):
    """A page table for the given numbers of positions, and how many pages there are."""
    r = np.random.RandomState(seed)
    cols = max(1, max((n + tokens - 1) // tokens for n in lengths))
    pages = len(lengths) * cols + spare
    table = torch.tensor(r.permutation(pages)[:len(lengths) * cols].reshape(len(lengths), cols), dtype=i32, device="cuda")
    return table, pages


def copy_of(cache):
    return [t.view(torch.uint8).clone().view(f8) if t.dtype == f8 else t.clone() for t in cache]


def assert_cache(got, want, what=""):
    for which in range(2):
        ref.assert_rounded(ref.values(got[which]), want.entry[which], f"{what} entries {which}")
        s = ref.doubles(got[2 + which])
        assert np.array_equal(s, want.scale[which]), f"{what} scales {which}"


@pytest.mark.parametrize("context,rows,heads,dim,tokens,block", [
    ([0], [1], 1, 64, 16, 16), ([0], [1], 2, 128, 64, 64), ([5], [1], 1, 128, 16, 1), ([15, 16, 17], [1, 1, 1], 2, 64, 16, 8),
    ([100, 3, 0], [6, 22, 2], 3, 128, 64, 16), ([130], [300], 2, 64, 32, 32), ([60, 64], [140, 1], 1, 128, 128, 128),
    ([1, 0, 255, 256], [3, 700, 2, 257], 2, 128, 256, 256), ([31], [33], 5, 64, 32, 2), ([9, 8, 7], [1, 2, 3], 2, 64, 16, 4)])
@pytest.mark.parametrize("dtype", [bf16, f32])
def test_cache_write_sizes(sv, context, rows, heads, dim, tokens, block, dtype):
    g = gen(sum(context) + sum(rows) + dim)
    table, pages = make_table(1, [c + n for c, n in zip(context, rows)], tokens)
    cache = make_cache(2, pages, heads, tokens, dim, block)
    spread = torch.exp(torch.randn(sum(rows), heads, 1, generator=g, device="cuda") * 2)
    k, v = ((torch.randn(sum(rows), heads, dim, generator=g, device="cuda") * spread).to(dtype) for _ in range(2))
    node_start = ints(0, *np.cumsum([n - 1 for n in rows]).tolist())
    want = ref.Cache(cache, table)
    want.write(k, v, ints(*context), node_start)
    sv.cache_write(cache, k, v, table, ints(*context), node_start)
    assert_cache(cache, want)


@pytest.mark.parametrize("order", ["head", "token"])
def test_cache_write_strides(sv, order):
    g = gen(4)
    context, rows, heads, dim, tokens, block = [7, 40], [12, 3], 3, 64, 16, 8
    table, pages = make_table(3, [19, 43], tokens)
    big = make_cache(5, pages, heads, tokens, dim, block, order=order)
    wide = torch.cat([table, table], 1)[:, :table.shape[1]]
    n = sum(rows)
    k = torch.randn(n, heads, dim + 3, generator=g, device="cuda")[:, :, 1:dim + 1]
    v = torch.randn(heads, n, dim, generator=g, device="cuda").transpose(0, 1)
    node_start = ints(0, rows[0] - 1, n - 2)
    want = ref.Cache(big, table)
    want.write(k, v, ints(*context), node_start)
    sv.cache_write(big, k, v, wide, ints(*context), node_start)
    assert_cache(big, want)


def test_cache_write_scales_grow_and_entries_follow(sv):
    # written one by one, louder and louder: each growth by a power of two moves no digits of the older entries
    heads, dim, tokens, block = 2, 64, 32, 32
    cache = make_cache(6, 3, heads, tokens, dim, block)
    table, g = ints(2, 0).view(1, 2), gen(7)
    rows = torch.randn(40, heads, dim, generator=g, device="cuda") * torch.exp2(torch.arange(40, device="cuda") / 4).view(-1, 1, 1)
    for p in range(40):
        want = ref.Cache(cache, table)
        want.write(rows[p:p + 1], -rows[p:p + 1], ints(p), ints(0, 0))
        sv.cache_write(cache, rows[p:p + 1], -rows[p:p + 1], table, ints(p), ints(0, 0))
        assert_cache(cache, want, p)
    k, v = ref.Cache(cache, table).sequence(0, 40)
    x = ref.doubles(rows).transpose(1, 0, 2)
    # half a step of an entry, and where a value has fallen below the smallest normal one 2^-10 of the scale for each of the
    # up to eight times that the scale grew
    size = np.repeat(ref.Cache(cache, table).scale[0][[2, 0]].transpose(1, 0, 2).reshape(heads, 2), 32, 1)[:, :40, None]
    assert np.all(np.abs(k - x) <= np.abs(x) * 2.0 ** -4 + 9 * 2.0 ** -10 * size)
    assert np.all(np.abs(v + x) <= np.abs(x) * 2.0 ** -4 + 9 * 2.0 ** -10 * size)


def test_cache_write_values_that_are_none_and_zeros(sv):
    heads, dim, tokens, block = 1, 64, 16, 16
    cache = make_cache(6, 2, heads, tokens, dim, block)
    table = ints(1).view(1, 1)
    k = torch.zeros(4, 1, dim, device="cuda")
    v = torch.randn(4, 1, dim, generator=gen(1), device="cuda")
    v[1, 0, 3], v[2, 0, 4], v[3, 0, 5] = float("nan"), float("inf"), float("-inf")
    want = ref.Cache(cache, table)
    want.write(k, v, ints(0), ints(0, 3))
    sv.cache_write(cache, k, v, table, ints(0), ints(0, 3))
    assert_cache(cache, want)
    assert float(cache[2][1, 0, 0]) == 2.0 ** -100
    tiny = torch.full((1, 1, dim), 1e-45, device="cuda")
    huge = torch.full((1, 1, dim), torch.finfo(f32).max, device="cuda")
    for x in (tiny, huge):
        want = ref.Cache(cache, table)
        want.write(x, x, ints(0), ints(0, 0))
        sv.cache_write(cache, x, x, table, ints(0), ints(0, 0))
        assert_cache(cache, want)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("offset", [0, 1])
def test_cache_write_values_that_are_none_anywhere_in_a_large_block(sv, dtype, offset):
    # in every quarter of a block, in every place of a run of eight, of either sign; rows without a finite value
    heads, dim, tokens, block, n = 2, 128, 256, 256, 250
    none = [float("nan"), float("inf"), float("-inf")]
    for at in range(0, n, 31):
        cache = make_cache(at, 2, heads, tokens, dim, block)
        table, g = ints(1).view(1, 1), gen(at)
        k, v = (torch.randn(n, heads, dim + offset, generator=g, device="cuda").to(dtype)[:, :, offset:] for _ in range(2))
        k[at, 0, at % dim] = none[at % 3]
        k[n - 1 - at, 1, (3 * at) % dim] = none[(at + 1) % 3]
        k[at, 1, 5] = -1e30
        v[:, 0] = none[at % 3]
        v[at] = none[(at + 2) % 3]
        want = ref.Cache(cache, table)
        want.write(k, v, ints(3), ints(0, n - 1))
        sv.cache_write(cache, k, v, table, ints(3), ints(0, n - 1))
        assert_cache(cache, want, at)


def test_cache_write_leaves_what_is_not_its_own(sv):
    # padded and invalid sequences, positions without pages
    heads, dim, tokens, block = 2, 64, 16, 8
    table, pages = make_table(3, [32] * 6, tokens)
    cache = make_cache(5, pages, heads, tokens, dim, block)
    sizes = [2, 20, 3, 2, 5, 1]
    node_start = ints(0, *np.cumsum(sizes).tolist())
    n = sum(sizes) + 6
    k, v = (torch.randn(n, heads, dim, generator=gen(i), device="cuda") for i in range(2))
    context = ints(-1, 14, 30, 0, 12, 2 ** 31 - 8)
    want = ref.Cache(cache, table)
    live = context.clone()
    live[0] = live[5] = -1
    # sequence 2: positions 30 to 33, of which 32 and 33 have no column; sequence 4: 12 to 17, of which 16 and 17 have no page
    spare = torch.full((6, 1), pages - 1, dtype=i32, device="cuda")  # stands in for the missing ones
    want.table = ref.ints(torch.cat([table, spare], 1))
    want.table[4, 1] = pages - 1
    kept = copy_of(cache)
    table[4, 1] = pages
    want.write(k, v, live, node_start)
    for which in range(2):
        want.entry[which][pages - 1] = ref.values(kept[which])[pages - 1]
        want.scale[which][pages - 1] = ref.doubles(kept[2 + which])[pages - 1]
    sv.cache_write(cache, k, v, table, context, node_start)
    assert_cache(cache, want)
    # ranges that are none, and more nodes than stated
    before = copy_of(cache)
    table[4, 1] = 0
    sv.cache_write(cache, k, v, table, torch.full((6,), 1, dtype=i32, device="cuda"), ints(5, 3, n, 2, -1, 9, -9))
    sv.cache_write(cache, k, v, table, ints(-1, 1, -1, -1, -1, -1), node_start, max_nodes=19)
    for a, b in zip(cache, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def rising_paths(seed, B, depth):
    """Paths that rise, of any length up to depth, and tokens' places of up to twice as many nodes."""
    r = np.random.RandomState(seed)
    path, length = np.full((B, depth), -1), r.randint(0, depth + 1, B)
    length[0], length[-1] = depth, 0
    for b in range(B):
        path[b, :length[b]] = np.sort(r.choice(2 * depth, length[b], replace=False))
    path[B // 2, :length[B // 2]] = np.arange(length[B // 2])  # one that moves nothing
    return torch.tensor(path, dtype=i32, device="cuda"), torch.tensor(length, dtype=i32, device="cuda")


@pytest.mark.parametrize("depth,B,heads,dim,tokens,block,layers", [
    (1, 2, 1, 64, 16, 16, None), (3, 5, 2, 128, 64, 32, None), (8, 7, 3, 64, 16, 8, 2), (5, 4, 1, 128, 32, 1, 3),
    (40, 6, 2, 128, 16, 16, None), (128, 3, 1, 64, 64, 64, None), (20, 5, 2, 64, 256, 128, 2), (33, 9, 1, 128, 128, 2, None)])
@pytest.mark.parametrize("order", ["head", "token"])
def test_cache_keep_sizes(sv, depth, B, heads, dim, tokens, block, layers, order):
    r = np.random.RandomState(depth + B)
    context = r.randint(0, 3 * tokens, B).tolist()
    context[0], context[-1] = tokens - 1, block - 1
    table, pages = make_table(depth, [c + 2 * depth + 1 for c in context], tokens)
    cache = make_cache(9, pages, heads, tokens, dim, block, layers, order)
    path, length = rising_paths(depth, B, depth)
    wants = [ref.Cache([t[i] for t in cache] if layers else cache, table) for i in range(layers or 1)]
    for w in wants:
        w.keep(path, length, ints(*context))
    got = sv.cache_keep(cache, path, length, table, ints(*context))
    assert torch.equal(got, ints(*context) + 1 + length)
    for i, w in enumerate(wants):
        assert_cache([t[i] for t in cache] if layers else cache, w, f"layer {i}")


def test_cache_keep_leaves_padded_and_invalid_sequences(sv):
    heads, dim, tokens, block, depth = 2, 64, 16, 16, 4
    table, pages = make_table(3, [40] * 9, tokens)
    cache = make_cache(5, pages, heads, tokens, dim, block)
    context = ints(-1, 3, 3, 3, 3, 46, 3, 14, 12)
    path = ints(*[1, 3, 4, 6] * 9).view(9, 4).contiguous()
    length = ints(2, -1, 5, 3, 2, 2, 2, 2, 3)
    path[3, 2] = 3  # does not rise
    path[4, 0] = -1
    # 5: no columns; 6: a page that is none
    table[6, 0] = -1
    table[7, 1] = pages  # position 15 is there, 16 and 18 are not
    before = copy_of(cache)
    got = sv.cache_keep(cache, path, length, table, context)
    keep_only_last = ref.Cache(before, table)
    c2, l2 = context.clone(), length.clone()
    l2[:8] = 0
    keep_only_last.keep(path, l2, c2)
    assert_cache(cache, keep_only_last)
    assert got.tolist() == [-1, 3, 3, 3, 3, 46, 3, 14, 16]


# ------------------------------------------------------------- attention

def attend_case(seed, context, sizes, heads, group, dim, tokens, block, order="head", chain=False):
    g = gen(seed)
    node_start, parent = random_trees(seed, sizes)
    table, pages = make_table(seed, [max(0, c) + n + 1 for c, n in zip(context, sizes)], tokens)
    cache = make_cache(seed + 1, pages, heads, tokens, dim, block, order=order)
    rows = int(sum(sizes)) + len(sizes)
    q = torch.randn(rows, heads * group, dim, generator=g, device="cuda").to(bf16)
    return dict(q=q, cache=cache, page_table=table, context=ints(*context), node_start=node_start,
                parent=None if chain else parent)


def assert_attends(got, c, scale=None, what="", rows=None):
    want, off = ref.Cache(c["cache"], c["page_table"]).attend(
        c["q"], c["context"], c["node_start"], c["parent"], c["q"].shape[2] ** -0.5 if scale is None else scale)
    have = ref.doubles(got)
    if rows is not None:
        want, off, have = want[rows], off[rows], have[rows]
    assert np.array_equal(np.isnan(have), np.isnan(want)), what
    fine = ~np.isnan(want)
    far = np.abs(have[fine] - want[fine])
    assert np.all(far <= off[fine]), (what, float(np.max(far / off[fine])))


@pytest.mark.parametrize("context,sizes", [
    ([0], [0]), ([1], [0]), ([127], [0]), ([128], [0]), ([126], [1]), ([129], [3]), ([0], [21]), ([0, 500, 3], [2, 0, 7]),
    ([255, 256, 257], [1, 1, 1]), ([1000], [60]), ([300, 0, 77, 128], [5, 5, 5, 5])])
@pytest.mark.parametrize("heads,group,dim,tokens,block", [(2, 4, 128, 64, 64), (1, 8, 64, 16, 16), (3, 1, 128, 128, 32)])
def test_attend_lengths(sv, context, sizes, heads, group, dim, tokens, block):
    c = attend_case(sum(context) + sum(sizes) + dim, context, sizes, heads, group, dim, tokens, block)
    assert_attends(sv.attend_tree(**c), c)


@pytest.mark.parametrize("heads,group,dim,tokens,block", [
    (1, 1, 64, 16, 1), (1, 2, 128, 32, 8), (2, 3, 64, 64, 16), (1, 5, 128, 256, 256), (4, 7, 64, 256, 64), (1, 16, 128, 16, 2),
    (2, 20, 64, 32, 32), (1, 33, 128, 64, 4), (1, 64, 64, 128, 128), (1, 71, 128, 64, 64)])
@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("order", ["head", "token"])
def test_attend_heads_pages_and_blocks(sv, heads, group, dim, tokens, block, chain, order):
    c = attend_case(heads * 100 + group, [200, 31], [9, 4], heads, group, dim, tokens, block, order, chain)
    assert_attends(sv.attend_tree(**c), c)


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("group,dim", [(1, 128), (4, 64)])
def test_attend_the_largest_tree(sv, chain, group, dim):
    c = attend_case(7, [130, 5], [256, 3], 1, group, dim, 64, 32, chain=chain)
    assert_attends(sv.attend_tree(**c), c)


@pytest.mark.parametrize("B", [40, 700])
def test_attend_many_sequences(sv, B):
    r = np.random.RandomState(B)
    context, sizes = r.randint(0, 300, B).tolist(), r.randint(0, 4, B).tolist()
    c = attend_case(B, context, sizes, 1, 2, 64, 32, 32)
    got = sv.attend_tree(**c)
    few = r.choice(B, 12, replace=False)
    rows = np.concatenate([np.arange(c["node_start"][b].item() + b, c["node_start"][b + 1].item() + b + 1) for b in few])
    c["context"][torch.tensor([b for b in range(B) if b not in set(few.tolist())], device="cuda")] = -1
    assert_attends(got, c, rows=rows)


@pytest.mark.parametrize("scale", [0.0, 0.3, -0.2, 3.0])
def test_attend_scales(sv, scale):
    # 3.0: a few positions take everything
    c = attend_case(3, [400], [4], 2, 2, 128, 64, 16)
    assert_attends(sv.attend_tree(**c, scale=scale), c, scale)


def test_attend_one_position_with_nearly_all_the_weight_and_many_with_the_rest(sv):
    # the first position of a long context takes a weight of 1, thousands of others less than 2^-12 each but most of the sum
    n, dim = 40000, 64
    c = attend_case(5, [n], [0], 1, 1, dim, 64, 64)
    k, v, ks, vs = c["cache"]
    ks.fill_(1.0), vs.fill_(1.0)
    first = int(c["page_table"][0, 0])
    k.view(torch.uint8)[:] = 0
    k.view(torch.uint8)[first, 0, 0] = 0x38  # ones
    q = torch.full_like(c["q"], 1.0)
    c["q"] = q * (9.0 / dim / dim ** -0.5)
    assert_attends(sv.attend_tree(**c), c)


@pytest.mark.parametrize("quiet", [1e-4, 1e4])
def test_attend_queries_and_keys_of_any_size(sv, quiet):
    # rows of one call that differ a million times in size, entries of a row that do
    c = attend_case(9, [300], [5], 1, 3, 128, 32, 8)
    g = gen(1)
    c["q"] = (c["q"].float() * torch.exp(torch.randn(c["q"].shape, generator=g, device="cuda") * 2) * quiet).to(bf16)
    c["cache"][2].mul_(1e-3 / quiet)
    c["q"][2] = 0
    c["q"][3, :, 1:] = 0
    assert_attends(sv.attend_tree(**c), c)


def test_attend_what_lies_behind_the_rows_or_beside_the_path_does_not_matter(sv):
    context, sizes = [100, 127, 60], [7, 3, 0]
    c = attend_case(21, context, sizes, 2, 2, 64, 16, 16)
    want = sv.attend_tree(**c).clone()
    k, v = (c["cache"][i].view(torch.uint8) for i in range(2))
    table = c["page_table"].tolist()
    for b, (n, m) in enumerate(zip(context, sizes)):
        for p in range(n + 1 + m, 16 * len(table[b])):
            k[table[b][p // 16], :, p % 16] = 0x7f
            v[table[b][p // 16], :, p % 16] = 0xff
    assert torch.equal(sv.attend_tree(**c), want)
    # NaN in a node's key, and in another's value: the rows that see them, and only they
    for t, node in ((k, 2), (v, 5)):
        p = context[0] + 1 + node
        t[table[0][p // 16], 1, p % 16, 3] = 0x7f
    got = sv.attend_tree(**c)
    parent = c["parent"].tolist()
    lost = [i for i in range(8) if {2, 5} & set(ref.path_of(parent, i))]
    assert 3 in lost and 6 in lost
    heads = slice(2, 4)
    others = [i for i in range(8) if i not in lost]
    assert bool(torch.isnan(got[lost][:, heads]).any(-1).all())
    keep = torch.ones(got.shape[:2], dtype=torch.bool, device="cuda")
    keep[lost, 2:4] = False
    assert torch.equal(got[keep], want[keep]) and others
    # in a committed place: every row of that head
    t = torch.isnan(got).any(-1)
    k[table[1][0], 0, 7, 0] = 0x7f
    assert bool(torch.isnan(sv.attend_tree(**c)[8 + 0:8 + 4, :2]).any(-1).all()) and not bool(t[8:].any())


def test_attend_queries_that_are_none(sv):
    c = attend_case(2, [200], [2], 1, 2, 128, 64, 64)
    want = sv.attend_tree(**c).clone()
    c["q"][0, 1, 5], c["q"][2, 0, 0] = float("nan"), float("inf")
    got = sv.attend_tree(**c)
    lost = torch.zeros(3, 2, dtype=torch.bool, device="cuda")
    lost[0, 1] = lost[2, 0] = True
    assert bool(torch.isnan(got[lost]).all()) and torch.equal(got[~lost], want[~lost])


def test_attend_padded_and_invalid_sequences(sv):
    sizes = [2, 3, 2, 2, 1]
    c = attend_case(4, [40, 90, 50, 33, 70], sizes, 1, 2, 64, 16, 16)
    want = sv.attend_tree(**c).clone()
    c["context"][0] = -1
    c["page_table"][1, 2] = len(c["cache"][0])
    c["parent"][5 + 1] = 1
    c["context"][3] = 2 ** 31 - 2
    out = torch.full_like(c["q"], 4.0)
    got = sv.attend_tree(**c, out=out)
    assert bool((got[:3] == 4).all()) and bool(torch.isnan(got[3:7]).all()) and bool(torch.isnan(got[7:10]).all())
    assert bool(torch.isnan(got[10:13]).all()) and torch.equal(got[13:], want[13:])
    # rows behind the last sequence, more nodes than stated, ranges that are none
    out = torch.full_like(c["q"], 4.0)
    got = sv.attend_tree(c["q"], c["cache"], c["page_table"], ints(40, 90, 50, 33, 70), ints(0, 2, 2, 50, 50, -1), None, out=out)
    assert bool((got[:3] != 4).any()) and bool((got[4:] == 4).all())
    out = torch.full_like(c["q"], 4.0)
    c["page_table"][1, 2] = 0
    got = sv.attend_tree(c["q"], c["cache"], c["page_table"], ints(40, 90, 50, 33, 70), c["node_start"], None, out=out, max_nodes=2)
    assert bool((got[3:7] == 4).all()) and not bool((got[7:] == 4).all(-1).any())


def test_attend_strides(sv):
    c = attend_case(6, [200, 17], [5, 2], 2, 3, 64, 32, 16)
    want = sv.attend_tree(**c)
    rows, H, D = c["q"].shape
    wide = torch.zeros(H, rows, D + 8, dtype=bf16, device="cuda")
    q = wide.transpose(0, 1)[..., :D]
    q.copy_(c["q"])
    store = torch.full((rows, H, D + 3), 7.0, dtype=bf16, device="cuda")
    got = sv.attend_tree(**dict(c, q=q), out=store[..., 1:D + 1])
    assert torch.equal(got, want)
    assert bool((store[..., 0] == 7).all()) and bool((store[..., D + 1:] == 7).all())
    # a table that is part of a wider one, a layer of a cache with layers in front
    layers = [torch.stack([t.view(torch.uint8), t.view(torch.uint8)]).view(f8) if t.dtype == f8 else torch.stack([t * 0, t])
              for t in c["cache"]]
    table = torch.cat([c["page_table"], torch.full_like(c["page_table"], -7)], 1)[:, :c["page_table"].shape[1]]
    import speculative_decoding_verification_online_gb300 as pkg
    got = sv.attend_tree(**dict(c, cache=pkg.PagedCache(*layers).layer(1), page_table=table))
    assert torch.equal(got, want)


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_a_cache_past_4_gb(sv, dim):
    tokens, heads = 256, 8
    pages = (5 << 30) // (tokens * heads * dim)
    c = attend_case(3, [700, 900], [3, 2], heads, 2, dim, tokens, 64)
    small = len(c["cache"][0])
    big = [torch.empty(pages, *t.shape[1:], dtype=torch.uint8 if t.dtype == f8 else t.dtype, device="cuda") for t in c["cache"]]
    at = torch.arange(small, device="cuda") * ((pages - 1) // (small - 1))
    for b, t in zip(big, c["cache"]):
        b[at] = t.view(torch.uint8) if t.dtype == f8 else t
    got = sv.attend_tree(**dict(c, cache=[b.view(f8) if b.dtype == torch.uint8 else b for b in big],
                                page_table=at[c["page_table"].long()].to(i32)))
    assert_attends(got, c)


def test_attend_long_contexts_are_split_and_joined(sv):
    context, sizes = [30000, 3, 9001], [4, 2, 0]
    c = attend_case(12, context, sizes, 1, 4, 64, 64, 64)
    assert_attends(sv.attend_tree(**c), c)


def test_attend_sequences_that_share_the_pages_of_a_prefix(sv):
    c = attend_case(12, [150, 131, 128, 400], [3, 0, 5, 2], 2, 4, 128, 64, 16)
    c["page_table"][:, :2] = c["page_table"][:1, :2].clone()
    assert_attends(sv.attend_tree(**c), c)


def test_attend_two_calls_at_once_with_the_same_inputs(sv):
    # on two streams, again and again: each has a workspace of its own
    c = attend_case(13, [3000, 77, 900], [9, 4, 0], 4, 4, 128, 64, 64)
    alone = sv.attend_tree(**c)
    assert_attends(alone, c)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(sv.attend_tree(**c))
    torch.cuda.synchronize()
    for out in outs[0] + outs[1]:
        assert torch.equal(out.view(torch.int16), alone.view(torch.int16))


def test_attend_is_deterministic(sv):
    c = attend_case(13, [5000, 700, 3000], [20, 3, 0], 2, 4, 128, 64, 16)
    first = sv.attend_tree(**c).clone()
    for _ in range(5):
        assert torch.equal(sv.attend_tree(**c), first)


# ------------------------------------------------------------- together

def step(sv, cache, s, stream=None):
    """One step of a tree's verification, as a program would make it: returns what it leaves."""
    kw = dict(stream=stream)
    sv.cache_write(cache, s["k"], s["v"], s["table"], s["context"], s["node_start"], max_nodes=s["most"], **kw)
    a = sv.attend_tree(s["q"], cache, s["table"], s["context"], s["node_start"], s["parent"], max_nodes=s["most"], **kw)
    logits = sv.linear(a.view(a.shape[0], -1), s["head"], out_dtype=f32, **kw)
    sv.penalize(logits, s["history"], s["history_len"], s["tokens"], s["parent"], s["node_start"], repetition=s["repetition"],
                frequency=s["frequency"], mask=s["mask"], mask_row=s["mask_row"], out=logits, **kw)
    p = sv.softmax(logits, 0.8, **kw)
    out = sv.verify_tree(p, None, s["tokens"], s["parent"], s["draft_row"], s["node_start"], s["u"], s["u_pick"],
                         max_nodes=s["most"], max_depth=s["depth"], **kw)
    context = sv.cache_keep(cache, out["path"], out["accepted_len"], s["table"], s["context"], **kw)
    return dict(out, attended=a, logits=logits, context=context)


def step_inputs(seed, B=5, heads=2, group=2, dim=64, V=700):
    g = gen(seed)
    sizes = [(seed + 3 * b) % 8 for b in range(B)]
    node_start, parent = random_trees(seed, sizes)
    total = sum(sizes)
    rows = total + B
    depth, par, at = 1, parent.tolist(), 0
    for n in sizes:
        for i in range(n):
            depth = max(depth, len(ref.path_of(par[at:at + n], i + 1)))
        at += n
    context = torch.randint(0, 150, (B,), generator=g, device="cuda").to(i32)
    table, pages = make_table(seed, [170] * B, 32)
    s = dict(node_start=node_start, parent=parent, most=8, depth=depth, context=context, table=table,
             tokens=torch.randint(0, 20, (total,), generator=g, device="cuda").to(i32),
             history=torch.randint(0, 30, (B, 60), generator=g, device="cuda").to(i32),
             history_len=torch.randint(0, 61, (B,), generator=g, device="cuda").to(i32),
             repetition=1.0 + torch.rand(B, generator=g, device="cuda"), frequency=torch.rand(B, generator=g, device="cuda") * 0.2,
             mask=torch.full((rows, 22), -1, dtype=i32, device="cuda"), mask_row=torch.arange(rows, device="cuda").to(i32),
             draft_row=torch.full((rows,), -1, dtype=i32, device="cuda"), u=torch.rand(total, generator=g, device="cuda") * 0.02,
             u_pick=torch.rand(B, generator=g, device="cuda"))
    s["mask"][:, 3] = 0x0f0f0f0f
    s["k"], s["v"] = (torch.randn(rows, heads, dim, generator=g, device="cuda").to(bf16) for _ in range(2))
    s["q"] = torch.randn(rows, heads * group, dim, generator=g, device="cuda").to(bf16)
    s["head"] = (torch.randn(V, heads * group * dim, generator=g, device="cuda") * 0.3).to(bf16)
    return s, make_cache(seed, pages, heads, 32, dim, 8)


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_a_step_of_verification(sv, seed):
    s, cache = step_inputs(seed)
    want = ref.Cache(cache, s["table"])
    out = step(sv, cache, s)
    want.write(s["k"], s["v"], s["context"], s["node_start"])
    for w in range(2):
        want.entry[w] = np.where(np.isnan(want.entry[w]), want.entry[w], _nearest(want.entry[w]))
    a, off = want.attend(s["q"], s["context"], s["node_start"], s["parent"], s["q"].shape[2] ** -0.5)
    assert np.all(np.abs(ref.doubles(out["attended"]) - a) <= off)
    z = out["attended"].view(len(a), -1).double() @ s["head"].double().T
    mag = out["attended"].view(len(a), -1).double().abs() @ s["head"].double().abs().T
    p, size = ref.penalties(z, s["history"], s["history_len"], s["tokens"], s["parent"], s["node_start"],
                            repetition=s["repetition"], frequency=s["frequency"], mask=s["mask"], mask_row=s["mask_row"])
    fine = np.isfinite(p)
    assert np.array_equal(fine, np.isfinite(ref.doubles(out["logits"])))
    # the product is off by 2^-17 of its magnitudes at most (64 steps of 2^-23), which a repetition may double
    bound = 2 * 2.0 ** -17 * ref.doubles(mag) + 20 * 2.0 ** -24 * (size + np.abs(np.where(fine, p, 0)))
    assert np.all(np.abs(ref.doubles(out["logits"]) - np.where(fine, p, 0))[fine] <= bound[fine])
    probs = sv.softmax(out["logits"], 0.8)
    walk, _ = op_ref.tree(ref.doubles(probs), None, *(s[k].cpu().numpy() for k in (
        "tokens", "parent", "draft_row", "node_start", "u", "u_pick")), 8, s["depth"])
    assert np.array_equal(walk["accepted_len"], out["accepted_len"].cpu().numpy())
    assert seed == 1 or walk["accepted_len"].max() > 0  # (the first one's trees are refused throughout)
    assert np.array_equal(walk["path"], out["path"].cpu().numpy())
    want.keep(out["path"], out["accepted_len"], s["context"])
    assert_cache(cache, want)
    assert torch.equal(out["context"], s["context"] + 1 + out["accepted_len"])


def _nearest(x):
    x = np.clip(x, -448.0, 448.0)
    at = np.clip(np.searchsorted(ref.FINITE, x), 1, len(ref.FINITE) - 1)
    lo, hi = ref.FINITE[at - 1], ref.FINITE[at]
    even = np.abs(x - lo) == np.abs(x - hi)
    step_ = hi - lo
    to_lo = np.where(even, np.round(lo / step_) % 2 == 0, np.abs(x - lo) < np.abs(x - hi))
    return np.where(to_lo, lo, hi)


def test_steps_captured_and_on_other_streams(sv):
    # two captured graphs and eager steps of the same inputs at once: the same results
    made = [step_inputs(seed) for seed in (4, 5)]
    wants = [step(sv, copy_of(cache), s) for s, cache in made]
    torch.cuda.synchronize()
    graphs, outs, caches = [], [], []
    for s, cache in made:
        own = copy_of(cache)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(sv, own, s))
        graphs.append(g)
        caches.append((own, cache))
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for own, cache in caches:
            for a, b in zip(own, cache):
                a.view(torch.uint8).copy_(b.view(torch.uint8))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        eager_cache = copy_of(made[0][1])
        streams[2].wait_stream(torch.cuda.current_stream())
        eager = step(sv, eager_cache, made[0][0], stream=streams[2])
        torch.cuda.synchronize()
        for want, got in zip(wants + wants[:1], outs + [eager]):
            for name in want:
                assert torch.equal(torch.nan_to_num(want[name].float()), torch.nan_to_num(got[name].float())), name
        for a, b in zip(eager_cache, caches[0][0]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("k", [1, 4])
def test_run_hidden_with_penalties_is_its_parts(sv, k):
    B, V, H = 6, 1500, 128
    g = gen(31)
    th, dh = (torch.randn(B, n, H, generator=g, device="cuda").to(bf16) for n in (k + 1, k))
    head = (torch.randn(V, H, generator=g, device="cuda") * 0.2).to(bf16)
    D = torch.randint(0, 40, (B, k), generator=g, device="cuda").to(i32)
    pen = dict(history=torch.randint(0, 60, (B, 50), generator=g, device="cuda").to(i32),
               history_len=torch.randint(0, 51, (B,), generator=g, device="cuda").to(i32),
               repetition=1.0 + torch.rand(B, generator=g, device="cuda"), presence=torch.rand(B, generator=g, device="cuda"))
    masks = [torch.full((B * n, (V + 31) // 32), -1, dtype=i32, device="cuda") for n in (k + 1, k)]
    for m in masks:
        m[:, 7] = 0
    ver = sv.SpecVerifier(B, k, V, device=0)
    try:
        got = ver.run_hidden(th, head, dh, head, D, 0.9, seed=3, logits_dtype=f32,
                             penalties=dict(pen, mask=masks[0], draft_mask=masks[1]))
        for name, hidden, n, m in (("target_logits", th, k + 1, masks[0]), ("draft_logits", dh, k, masks[1])):
            z = sv.linear(hidden.reshape(B * n, H), head, out_dtype=f32)
            nodes = D[:, :n - 1].contiguous()
            start = ints(*range(0, B * (n - 1) + 1, n - 1)) if n > 1 else torch.zeros(B + 1, dtype=i32, device="cuda")
            want, size = ref.penalties(z, tokens=nodes.view(-1), parent=None, node_start=start, mask=m, **pen)
            have = ref.doubles(got[name].view(B * n, V))
            fine = np.isfinite(want)
            assert np.array_equal(fine, np.isfinite(have)) and not fine[:, 7 * 32].any()
            assert np.all(np.abs(have[fine] - want[fine]) <= 20 * 2.0 ** -24 * (size + np.abs(want))[fine])
        again = ver.run(got["target_logits"], got["draft_logits"], D, 0.9, seed=3)
        assert torch.equal(again["tokens"], got["tokens"])
    finally:
        ver.close()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group,nodes", [(1, 3), (4, 0), (8, 0), (3, 2), (4, 3), (5, 4), (8, 2), (6, 4), (8, 4), (4, 12), (7, 8)])
def test_attend_as_many_columns_as_a_call_may_need(sv, dim, group, nodes):
    # 4 to 64 columns of a key head: each of the kernel's widths, with sequences that fill it and others that do not
    sizes = [nodes, 0, max(0, nodes - 1), nodes]
    c = attend_case(group * 31 + nodes, [700, 1, 130, 3000], sizes, 2, group, dim, 64, 32)
    assert_attends(sv.attend_tree(**c), c)


def test_attend_values_scales_of_any_size(sv):
    # scales that differ from position to position, a million times, zeros among them; and blocks whose values are all zero
    c = attend_case(17, [900, 40], [5, 2], 1, 4, 128, 64, 1)
    g = gen(8)
    vs = c["cache"][3]
    vs.mul_(torch.exp(torch.randn(vs.shape, generator=g, device="cuda") * 3))
    vs[torch.rand(vs.shape, generator=g, device="cuda") < 0.1] = 2.0 ** -100
    assert_attends(sv.attend_tree(**c), c)
    vs.fill_(2.0 ** -100)
    assert_attends(sv.attend_tree(**c), c)
