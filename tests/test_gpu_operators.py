"""The operators around a verifying call on the GPU: matrix products, row
probabilities and tree verification against 64-bit implementations, and a run
of them together.  Token ids have to be equal, everything else within bounds
derived beside it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import oracle as O
from tests import operators_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verification_online_gb300 as pkg
    from speculative_decoding_verification_online_gb300 import build as B
    B.build()
    pkg.load()
    return pkg


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------- linear

def _operands(seed, G, M, N, K, shared=False, pad=0, offset=0):
    g = _gen(seed)

    def rows(n_rows, k):
        store = torch.full((offset + n_rows * (k + pad),), float("nan"), dtype=torch.bfloat16, device="cuda")
        v = store[offset:].view(n_rows, k + pad)[:, :k]
        v.copy_(torch.randn(n_rows, k, generator=g, device="cuda"))
        return v

    x = rows((1 if shared else G) * M, K)
    w = rows(G * N, K)
    x = x if shared else x.unflatten(0, (G, M))
    return x, w.unflatten(0, (G, N)), g


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 64), (1, 4096, 512), (2, 130, 72), (5, 127, 63), (16, 256, 128), (17, 129, 200),
    (33, 384, 1024), (64, 1000, 320), (77, 515, 1001), (96, 640, 136), (128, 128, 4096), (129, 257, 65), (200, 300, 96),
    (256, 512, 512), (257, 513, 520), (384, 1280, 256), (511, 100, 48), (640, 2048, 384)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_linear_sizes(sv, M, N, K, out):
    x, w, g = _operands(M * 7 + N, 1, M, N, K)
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    y = sv.linear(x[0], w[0], out_dtype=dt)
    assert y.dtype == dt and y.shape == (M, N)
    ref.assert_linear(y, x[0], w[0], None, None, "none", 0.0, f"{M}x{N}x{K}")


@pytest.mark.parametrize("M,N,K", [(1, 500, 8192), (6, 2000, 4100), (100, 300, 3001), (128, 160, 2048), (200, 700, 8192),
                                   (384, 512, 1030), (150, 300, 2049), (7, 500, 1536), (130, 600, 1537), (77, 900, 1001), (300, 500, 1280), (40, 64, 769), (300, 64, 768)])
def test_linear_long_sums_in_fp32(sv, M, N, K):
    # Whatever K, at most 48 steps of 16 products go into one sum of the tensor core, and 48 + 16 where halves of K are
    # rounded up to whole stages: K <= 768 in one, up to 1536 in two, longer ones in segments of 512, added in fp32.  A step is off by less than 2^-23 of the sums of |x w| for each of
    # its 16 products and itself.
    x, w, g = _operands(M + K, 1, M, N, K)
    x, w = x[0], w[0]
    y = sv.linear(x, w, out_dtype=torch.float32)
    want, mag = x.double() @ w.double().T, x.double().abs() @ w.double().abs().T
    off = (y.double() - want).abs()
    assert bool((off <= (64 * 2.0 ** -23 + K / 512 * 2.0 ** -24) * mag).all())
    # a sum of n steps that each cut off half a step on the average: n / 2 * 2^-23 in the 2-norm at most
    assert float(off.norm() / want.norm()) <= 32 * 2.0 ** -23
    ref.assert_linear(y, x, w, None, None, "none", 0.0)


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "softcap"])
@pytest.mark.parametrize("M,N,K", [(3, 200, 64), (70, 333, 257), (300, 512, 128)])
def test_linear_epilogues(sv, act, M, N, K):
    x, w, g = _operands(M + len(act), 1, M, N, K)
    x, w = x[0], w[0]
    for bdt, rdt, ydt in ((torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.float32, torch.bfloat16, torch.float32),
                          (torch.bfloat16, torch.float32, torch.bfloat16), (None, torch.float32, torch.float32),
                          (torch.float32, None, torch.bfloat16)):
        bias = None if bdt is None else torch.randn(N, generator=g, device="cuda").to(bdt) * 3
        res = None if rdt is None else torch.randn(M, N, generator=g, device="cuda").to(rdt)
        y = sv.linear(x, w, bias=bias, residual=res, activation=act, cap=5.0, out_dtype=ydt)
        ref.assert_linear(y, x, w, bias, res, act, 5.0, f"{act} {bdt} {rdt} {ydt}")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh", "softcap"])
@pytest.mark.parametrize("M", [1, 200])
def test_linear_activations_over_their_range(sv, act, M):
    # without entries of K an activation's argument is the bias itself
    z = torch.cat([torch.linspace(-40, 40, 20001), torch.logspace(-30, 30, 5000), -torch.logspace(-30, 30, 5000),
                   torch.tensor([0.0, -0.0, float("inf"), float("-inf"), float("nan")])]).cuda()
    empty = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda")
    y = sv.linear(empty, torch.empty(len(z), 0, dtype=torch.bfloat16, device="cuda"), bias=z, activation=act, cap=5.0,
                  out_dtype=torch.float32)
    finite = z.isfinite()
    assert torch.equal(y[:, finite], y[:1, finite].expand(M, -1))
    ref.assert_linear(y[:, finite], empty, torch.empty(int(finite.sum()), 0, device="cuda"), z[finite], None, act, 5.0, act)
    want = ref.ACT[act](z[~finite].double(), 5.0)
    assert torch.equal(torch.isnan(y[:, ~finite]), torch.isnan(want).expand(M, -1))
    there = ~torch.isnan(want)
    assert torch.equal(y[:, ~finite][:, there].double(), want[there].expand(M, -1))


@pytest.mark.parametrize("G,M,N,K,shared,pad,offset", [
    (4, 1, 512, 256, True, 0, 0), (5, 6, 384, 512, True, 8, 0), (3, 17, 200, 100, False, 0, 0),
    (2, 77, 321, 129, False, 3, 1), (5, 64, 256, 320, False, 8, 8), (2, 130, 140, 72, True, 1, 0),
    (7, 300, 128, 64, False, 0, 4)])
def test_linear_groups_strides_and_layouts(sv, G, M, N, K, shared, pad, offset):
    x, w, g = _operands(G * 100 + M, G, M, N, K, shared, pad, offset)
    bias = torch.randn(G, N + 5, generator=g, device="cuda")[:, 2:2 + N]
    res = torch.randn(M, G, N, generator=g, device="cuda").to(torch.bfloat16).transpose(0, 1)
    store = torch.full((M, G, N + 2), 7.0, device="cuda")
    out = store[:, :, 1:N + 1].transpose(0, 1)
    y = sv.linear(x, w, bias=bias, residual=res, activation="silu", out=out)
    assert y is out
    ref.assert_linear(out, x, w, bias, res, "silu", 0.0)
    assert bool((store[:, :, 0] == 7).all()) and bool((store[:, :, -1] == 7).all())  # nothing beside the rows


# rows, groups and the first entry at every place in 16 bytes; classes of rows that are empty, one row, one row more than a
# tile; more groups than places; rows that overlap; several tiles of tokens
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("G,M,N,K,row,group,offset", [
    (1, 5, 1, 70, 75, 0, 3), (1, 9, 3, 1, 5, 0, 1), (2, 4, 9, 64, 65, 593, 7), (3, 33, 17, 57, 61, 1041, 6),
    (1, 20, 2049, 130, 133, 0, 5), (1, 130, 129, 200, 203, 0, 2), (17, 3, 40, 90, 91, 3645, 1), (9, 6, 50, 128, 132, 6603, 4),
    (5, 2, 30, 65, 66, 1981, 0), (1, 300, 520, 1000, 1002, 0, 1), (2, 257, 100, 1100, 1101, 110107, 3),
    (1, 129, 1030, 1601, 1603, 0, 7), (1, 40, 60, 100, 7, 0, 1), (4, 8, 24, 320, 320, 7681, 0), (3, 260, 80, 96, 96, 0, 1),
    (2, 1, 4100, 2001, 2001, 8204100, 0), (3, 64, 1025, 63, 63, 64577, 5)])
def test_linear_reads_nothing_beside_its_rows(sv, G, M, N, K, row, group, offset, out):
    g = _gen(M * N + K)

    def operand(groups, rows, row, group, offset):
        store = torch.full((offset + (groups - 1) * group + (rows - 1) * row + K + 16,), float("nan"), dtype=torch.bfloat16,
                           device="cuda")
        view = torch.as_strided(store, (groups, rows, K), (group, row, 1), offset)
        for i in range(groups):
            for r in range(rows) if row < K else (slice(None),):  # rows that overlap: one after the other
                part = view[i, r]
                part.copy_(torch.randn(part.shape, generator=g, device="cuda") / K ** 0.5)
        return view

    w = operand(G, N, row, group, offset)
    for x in (operand(1, M, K + 3, 0, 1)[0], operand(1, M, (K + 7) // 8 * 8, 0, 0)[0],
              operand(G, M, K + 1, M * (K + 1) + 5, 6)):
        res = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16).expand(G, M, N)
        bias = torch.randn(G, N, generator=g, device="cuda")
        y = sv.linear(x, w, bias=bias, residual=res, activation="gelu",
                      out_dtype=torch.bfloat16 if out == "bf16" else torch.float32)
        ref.assert_linear(y, x, w, bias, res, "gelu", 0.0)


# tiles wider than half of the finishing threads, few tokens and one more than few
@pytest.mark.parametrize("M", [1, 4, 5, 20, 32, 33])
@pytest.mark.parametrize("N,K", [(40001, 72), (40001, 75), (40000, 800), (30007, 1601)])
def test_linear_few_tokens_wide_tiles(sv, M, N, K):
    x, w, g = _operands(M + K, 1, M, N, K)
    x, w = x[0], w[0]
    res = torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16)
    bias = torch.randn(N, generator=g, device="cuda")
    for b, r, act, ydt in ((None, None, "none", torch.bfloat16), (bias, res, "gelu", torch.float32),
                           (bias, None, "softcap", torch.float32), (None, res, "silu", torch.bfloat16)):
        store = torch.full((M, N + 2), 7.0, device="cuda").to(ydt)
        sv.linear(x, w, bias=b, residual=r, activation=act, cap=5.0, out=store[:, 1:N + 1])
        ref.assert_linear(store[:, 1:N + 1], x, w, b, r, act, 5.0, act)
        assert bool((store[:, 0] == 7).all()) and bool((store[:, -1] == 7).all())


def test_linear_into_its_own_residual(sv):
    x, w, g = _operands(3, 1, 70, 260, 192)
    res = torch.randn(70, 260, generator=g, device="cuda").to(torch.bfloat16)
    out = res.clone()
    sv.linear(x[0], w[0], residual=out, activation="silu", out=out)
    ref.assert_linear(out, x[0], w[0], None, res, "silu", 0.0)


def test_linear_empty_sizes(sv):
    x, w, g = _operands(3, 2, 5, 40, 16)
    bias, res = torch.randn(2, 40, device="cuda"), torch.randn(2, 5, 40, device="cuda")
    y = sv.linear(x[:, :, :0], w[:, :, :0], bias=bias, residual=res, activation="relu", out_dtype=torch.float32)
    assert torch.equal(y, bias.unsqueeze(1).clamp(min=0) + res)
    assert sv.linear(x[:, :0], w).shape == (2, 0, 40)
    assert sv.linear(x, w[:, :0]).shape == (2, 5, 0)
    assert sv.linear(x[:0], w[:0]).shape == (0, 5, 40)


def test_linear_keeps_infinities_and_nan_where_they_are(sv):
    x, w, g = _operands(5, 1, 40, 300, 128)
    x, w = x[0].clone(), w[0].clone()
    x[3, 7] = float("inf")
    x[9, 100] = float("nan")
    w[17, 5] = float("-inf")
    w[:, 7] = w[:, 7].abs() + 0.5
    y = sv.linear(x, w, out_dtype=torch.float32)
    want = x.double() @ w.double().T
    assert bool((torch.isnan(y) == torch.isnan(want)).all())
    at = torch.isinf(want)
    assert bool((y.double()[at] == want[at]).all()) and bool((torch.isinf(y) == at).all())


def test_linear_is_deterministic_and_replays(sv):
    x, w, g = _operands(8, 4, 3, 1024, 2048, shared=True)
    first = sv.linear(x, w, out_dtype=torch.float32)
    assert all(torch.equal(first, sv.linear(x, w, out_dtype=torch.float32)) for _ in range(5))
    out = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.linear(x, w, out=out)
    for i in range(2):
        x.normal_(generator=g)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, sv.linear(x, w, out_dtype=torch.float32))


def test_linear_large_offsets(sv):
    # the last rows of w and y start past 2^31 elements
    n_far, K = 40, 128
    w = torch.empty((1 << 31) + 4096 * K, dtype=torch.bfloat16, device="cuda")
    stride = ((1 << 31) // (n_far - 1) // 8 + 1) * 8
    view = torch.as_strided(w, (n_far, K), (stride, 1))
    x, wv, g = _operands(4, 1, 20, n_far, K)
    view.copy_(wv[0])
    y = torch.as_strided(torch.empty((1 << 31) + 4096, device="cuda"), (20, n_far), ((1 << 31) // 19, 1))
    sv.linear(x[0], view, out=y)
    ref.assert_linear(y, x[0], wv[0], None, None, "none", 0.0)


@pytest.mark.parametrize("M", [20, 140])
def test_linear_large_offsets_at_odd_addresses(sv, M):
    # rows of both operands past 2^31 elements, at every place in 16 bytes
    n_far, K = 40, 201
    stride = (1 << 31) // (n_far - 1) // 8 * 8 + 9
    w = torch.as_strided(torch.empty(stride * n_far, dtype=torch.bfloat16, device="cuda"), (n_far, K), (stride, 1), 3)
    xs = (1 << 31) // (M - 1) // 8 * 8 + 13
    x = torch.as_strided(torch.empty(xs * M, dtype=torch.bfloat16, device="cuda"), (M, K), (xs, 1), 1)
    xv, wv, g = _operands(4, 1, M, n_far, K)
    x.copy_(xv[0]), w.copy_(wv[0])
    ref.assert_linear(sv.linear(x, w, out_dtype=torch.float32), xv[0], wv[0], None, None, "none", 0.0)


def test_linear_rows_that_share_their_place(sv):
    # operands whose rows or groups are one (strides of 0), as expand leaves them
    g = _gen(12)
    row = torch.randn(1, 192, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(3, 300, 192, generator=g, device="cuda").to(torch.bfloat16)
    res = torch.randn(1, 300, generator=g, device="cuda").to(torch.bfloat16)
    for M in (5, 150):
        x = row.expand(M, 192)
        y = sv.linear(x, w, residual=res.expand(3, M, 300), bias=res[0].expand(3, 300), out_dtype=torch.float32)
        ref.assert_linear(y, x, w, res[0].expand(3, 300), res.expand(3, M, 300), "none", 0.0)
        same = sv.linear(x.expand(3, M, 192), w[:1].expand(3, 300, 192), out_dtype=torch.float32)
        ref.assert_linear(same, x, w[:1].expand(3, 300, 192), None, None, "none", 0.0)


@pytest.mark.parametrize("M", [3, 200])
def test_linear_without_entries_of_k_over_many_tiles(sv, M):
    bias = torch.randn(4, 20000, generator=_gen(M), device="cuda")
    empty = torch.empty(4, 20000, 0, dtype=torch.bfloat16, device="cuda")
    y = sv.linear(empty[0, :M], empty, bias=bias, activation="relu", out_dtype=torch.float32)
    assert torch.equal(y, bias.clamp(min=0).unsqueeze(1).expand(4, M, 20000))


def test_calls_at_once_on_two_streams(sv):
    # eager calls of every operator and a replayed capture of them, side by side
    x, w, g = _operands(14, 2, 200, 1000, 512)
    xs, ws, _ = _operands(15, 4, 2, 700, 1032, shared=True, pad=3)
    logits = torch.randn(60, 50000, generator=g, device="cuda").to(torch.bfloat16)
    t = ref.on_gpu(ref.random_tree_batch(24, 16, 20000, 5, 5, True, "mixed", noise=1.0))
    tree = [t[k] for k in ("p", "q", "tokens", "parent", "draft_row", "node_start", "u_accept", "u_pick")]

    def all_of_them():
        out = sv.verify_tree(*tree, max_nodes=5, max_depth=5)
        return [sv.linear(x, w, out_dtype=torch.float32), sv.linear(xs, ws), sv.softmax(logits, 0.8)] + \
            [out[k] for k in sorted(out)]

    want = all_of_them()
    torch.cuda.synchronize()
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=one):
        captured = all_of_them()
    got = []
    for _ in range(8):
        with torch.cuda.stream(one):
            graph.replay()
        with torch.cuda.stream(two):
            got.append(all_of_them())
    torch.cuda.synchronize()
    for result in got + [captured]:
        for a, b in zip(result, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------- softmax

def _assert_softmax(got, logits, t):
    """An exponent's argument a (in powers of two) is off by 4 half steps of itself, so exp2 by 4 ln 2 |a| of them;
    exp2 by 4 and the division and product by 2 more; a sum of V terms in runs of at most V / 256 + 32 additions."""
    V = logits.shape[1]
    t = t if isinstance(t, float) else t.double().unsqueeze(1)
    z = logits.double() / t
    want = torch.softmax(z, 1)
    a = (z - z.amax(1, keepdim=True)).abs() * 1.4427
    mean_a = (want * a).sum(1, keepdim=True)  # the sum's own error from its terms' arguments
    steps = 4 * 0.7 * (a + mean_a) + 16 + V / 256 + 32
    bound = steps * 2.0 ** -24 * want + 2.0 ** -126
    off = (got.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V", [(1, 1), (3, 2), (5, 7), (2, 1023), (4, 1024), (1, 4097), (9, 32000), (2, 128256),
                                    (1, 262143), (700, 2049), (3, 65537), (40, 50001)])
def test_softmax_sizes(sv, dtype, rows, V):
    g = _gen(rows + V)
    x = (torch.randn(rows, V, generator=g, device="cuda") * 4).to(dtype)
    _assert_softmax(sv.softmax(x, 0.7), x, 0.7)
    t = torch.rand(rows, generator=g, device="cuda") + 0.3
    _assert_softmax(sv.softmax(x, t), x, t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(1, 0), (3, 1), (8, 0), (4, 2)])
def test_softmax_strides_and_alignment(sv, dtype, pad, offset):
    rows, V = 6, 3001
    store = torch.full((offset + rows * (V + pad),), float("nan"), dtype=dtype, device="cuda")
    x = store[offset:].view(rows, V + pad)[:, :V]
    x.copy_(torch.randn(rows, V, generator=_gen(pad), device="cuda"))
    out_store = torch.full((rows, V + 2 * pad), 9.0, device="cuda")
    out = out_store[:, pad:pad + V]
    sv.softmax(x, 1.3, out=out)
    _assert_softmax(out, x, 1.3)
    assert bool((out_store[:, :pad] == 9).all()) and bool((out_store[:, pad + V:] == 9).all())


def test_softmax_temperature_zero_takes_the_first_largest(sv):
    x = torch.randn(5, 40000, generator=_gen(1), device="cuda").to(torch.bfloat16)
    x[1, 30000] = x[1, 5] = 50.0
    x[2] = 1.0
    x[3] = float("-inf")
    x[3, 39999] = -3.0e38
    x[4, 7:] = float("-inf")
    y = sv.softmax(x, 0.0)
    want = torch.zeros_like(y)
    want[torch.arange(5), x.float().argmax(1)] = 1
    want[1] = 0
    want[1, 5] = 1
    want[2] = 0
    want[2, 0] = 1
    assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [10, 5000, 140000])
def test_softmax_rows_without_a_distribution(sv, dtype, V):
    x = torch.randn(9, V, generator=_gen(V), device="cuda").to(dtype)
    x[1, V - 1] = float("nan")
    x[2, V // 2] = float("inf")
    x[3] = float("-inf")
    x[4, : V - 1] = float("-inf")
    x[5] = torch.finfo(dtype).min
    t = torch.ones(9, device="cuda")
    t[6], t[7], t[8] = -1.0, float("nan"), float("inf")
    y = sv.softmax(x, t)
    assert bool(torch.isnan(y[[1, 2, 3, 6, 7, 8]]).all())
    cold = sv.softmax(x, torch.where(t > 0, 0.0, t))
    assert bool(torch.isnan(cold[[1, 2, 3, 6, 7]]).all())
    assert torch.equal(cold[[0, 4, 5]].argmax(1), x[[0, 4, 5]].float().argmax(1))
    assert bool((cold[[0, 4, 5]].sum(1) == 1).all())
    mixed = sv.softmax(x, torch.tensor([0.0, 1, 0, 1, 1, 1, 0, 0, 1], device="cuda"))  # warm and cold rows in turn
    assert torch.equal(mixed[[0, 4]], torch.cat([cold[:1], y[4:5]]))
    assert torch.equal(y[4], torch.nn.functional.one_hot(torch.tensor(V - 1), V).float().cuda())
    _assert_softmax(y[[0, 5]], x[[0, 5]], 1.0)


def test_softmax_in_place_and_empty(sv):
    x = torch.randn(7, 30000, generator=_gen(2), device="cuda")
    before = x.clone()
    sv.softmax(x, 0.9, out=x)
    _assert_softmax(x, before, 0.9)
    assert sv.softmax(x[:0], 1.0).shape == (0, 30000)


# ------------------------------------------------------------- tree

def _run_tree(sv, batch, max_nodes, max_depth, replacement=True, pad=0, offset=0, **kw):
    t = ref.on_gpu(batch, pad, offset)
    cnt = torch.zeros(8, dtype=torch.int64, device="cuda")
    out = sv.verify_tree(t["p"], t["q"], t["tokens"], t["parent"], t["draft_row"], t["node_start"], t["u_accept"],
                         t["u_pick"], max_nodes=max_nodes, max_depth=max_depth, replacement=replacement, counters=cnt,
                         **kw)
    torch.cuda.synchronize()
    return {k: v.cpu().numpy() for k, v in out.items()}, cnt.cpu().numpy()


def _assert_tree(got, want):
    (g, gc), (w, wc) = got, want
    for name in ("accepted_len", "tokens", "path", "flags"):
        assert np.array_equal(g[name], w[name]), (name, np.argwhere(g[name] != w[name])[:5])
    # one rounding to fp32 of a value good to 1e-12
    np.testing.assert_allclose(g["accept_prob"], w["accept_prob"], rtol=2.0 ** -24 + 1e-9, atol=1e-30)
    assert np.array_equal(gc, wc), (gc, wc)


def _check_tree(sv, batch, max_nodes, max_depth, replacement=True, **kw):
    want = ref.tree(batch["p"], batch["q"], batch["tokens"], batch["parent"], batch["draft_row"], batch["node_start"],
                    batch["u_accept"], batch["u_pick"], max_nodes, max_depth, replacement)
    _assert_tree(_run_tree(sv, batch, max_nodes, max_depth, replacement, **kw), want)
    return want


@pytest.mark.parametrize("replacement", [True, False])
@pytest.mark.parametrize("kind", ["sampled", "mixed", "certain"])
@pytest.mark.parametrize("V", [1, 2, 7, 67, 1000, 1024, 1025, 5000])
def test_tree_random(sv, V, kind, replacement):
    batch = ref.random_tree_batch(V + 17 * replacement + len(kind), 40, V, 12, 5, replacement, kind, noise=1.2)
    w, cnt = _check_tree(sv, batch, 12, 5, replacement)
    if V > 2 and (kind != "certain" or V < 100):  # certain proposals of a flat long row are hardly ever accepted
        assert cnt[1] > 0 and cnt[3] > 0 and cnt[4] > 0


@pytest.mark.parametrize("V,B", [(32000, 3), (128256, 2), (151936, 1), (262144, 1), (40001, 20), (9000, 170)])
def test_tree_large_vocabularies(sv, V, B):
    batch = ref.random_tree_batch(V, B, V, 5, 3, True, "mixed", sharp=3.0, noise=1.0)
    _check_tree(sv, batch, 5, 3)


@pytest.mark.parametrize("pad,offset", [(0, 1), (1, 0), (3, 2), (4, 0), (8, 4)])
def test_tree_strides_and_alignment(sv, pad, offset):
    batch = ref.random_tree_batch(pad * 10 + offset, 12, 3003, 8, 4, False, "mixed", noise=1.2)
    _check_tree(sv, batch, 8, 4, False, pad=pad, offset=offset)


def test_tree_chains_stars_and_the_largest_tree(sv):
    _check_tree(sv, ref.random_tree_batch(1, 6, 50, 256, 256, True, "sampled", noise=0.05, shape="chain"), 256, 256)
    _check_tree(sv, ref.random_tree_batch(2, 6, 300, 256, 256, True, "sampled", noise=3.0, shape="star"), 256, 256)
    _check_tree(sv, ref.random_tree_batch(3, 6, 300, 256, 256, False, "sampled", noise=3.0, shape="star"), 256, 1, False)
    _check_tree(sv, ref.random_tree_batch(4, 6, 300, 256, 256, True, "certain", shape="star"), 256, 1)
    _check_tree(sv, ref.random_tree_batch(5, 30, 300, 256, 9, True, "mixed", noise=1.0), 256, 9)


def test_tree_without_nodes_samples_the_root(sv):
    batch = ref.random_tree_batch(7, 33, 999, 0, 0, True)
    w, cnt = _check_tree(sv, batch, 0, 0)
    assert cnt[4] == 33
    batch["q"] = np.zeros((0, 999), np.float32)
    batch["draft_row"][:] = -1
    _check_tree(sv, batch, 0, 0)


def test_tree_ties_and_extreme_uniforms(sv):
    # dyadic rows: every comparison is an equality somewhere, and exact in any order
    rng = np.random.default_rng(3)
    batch = ref.random_tree_batch(9, 200, 64, 6, 4, True, "mixed")
    R = batch["p"].shape[0]
    for name in ("p", "q"):
        w = rng.multinomial(64, np.ones(64) / 64, R) / 64.0
        batch[name] = w.astype(np.float32)
    batch["u_accept"] = (rng.integers(0, 8, len(batch["u_accept"])) / 8).astype(np.float32)
    batch["u_pick"] = (rng.integers(0, 16, 200) / 16).astype(np.float32)
    batch["u_pick"][:20], batch["u_pick"][20:40] = 0.0, 1 - 2.0 ** -24
    _check_tree(sv, batch, 6, 4)


def test_tree_rows_with_zeros_and_no_mass(sv):
    # rows that need not be normalised: rests without mass fall back to p, rows without mass are invalid
    batch = ref.random_tree_batch(11, 64, 40, 4, 3, True, "mixed", shape="any")
    rng = np.random.default_rng(4)
    batch["p"] *= (rng.random(batch["p"].shape) < 0.3)
    batch["q"] = np.where(rng.random(batch["q"].shape[0])[:, None] < 0.5, np.float32(1.0), batch["q"]).astype(np.float32)
    batch["p"][batch["node_start"][5] + 5] = 0.0  # the root of sequence 5
    w, cnt = _check_tree(sv, batch, 4, 3)
    assert cnt[7] > 0 and cnt[6] > 0


def test_tree_invalid_sequences_fail_closed(sv):
    batch = ref.random_tree_batch(13, 20, 500, 6, 6, True, "sampled")
    st = batch["node_start"]
    has = [b for b in range(20) if st[b + 1] - st[b] >= 3]
    assert len(has) >= 6
    batch["tokens"][st[has[0]] + 1] = 500
    batch["tokens"][st[has[1]] + 2] = -1
    batch["parent"][st[has[2]] + 1] = 1
    batch["parent"][st[has[3]]] = -2
    batch["draft_row"][st[has[4]] + has[4]] = batch["q"].shape[0]
    batch["draft_row"][st[has[5]] + has[5] + 1] = -7
    w, cnt = _check_tree(sv, batch, 6, 6)
    assert cnt[6] == 6
    # too deep, too many nodes, ranges that leave the arrays
    chain = ref.random_tree_batch(14, 8, 100, 6, 6, True, shape="chain")
    w, cnt = _check_tree(sv, chain, 6, 3)
    assert cnt[6] > 0
    w, cnt = _check_tree(sv, chain, 4, 4)
    assert cnt[6] > 0
    for bad in (-1, 1 << 30, -(1 << 31)):
        broken = dict(chain, node_start=chain["node_start"].copy())
        broken["node_start"][3] = bad
        got, gc = _run_tree(sv, broken, 6, 6)
        assert got["accepted_len"][2] == -1 and got["accepted_len"][3] == -1
        assert (got["tokens"][2:4] == -1).all() and (got["path"][2:4] == -1).all()
        keep = [0, 1, 4, 5, 6, 7]
        want = ref.tree(*(chain[k] for k in ("p", "q", "tokens", "parent", "draft_row", "node_start", "u_accept",
                                             "u_pick")), 6, 6)[0]
        assert np.array_equal(got["tokens"][keep], want["tokens"][keep])


@pytest.mark.parametrize("what", ["nan_p", "inf_p", "nan_q", "nan_p_unread"])
def test_tree_probabilities_that_are_none(sv, what):
    batch = ref.random_tree_batch(15, 30, 3000, 3, 3, True, "sampled", shape="chain")
    if what == "nan_p":
        batch["p"][:, 2999] = np.nan
    elif what == "inf_p":
        batch["p"][:, 1500] = np.inf
    elif what == "nan_q":
        batch["q"][:, 17] = np.nan
    else:
        batch["p"][batch["node_start"][5] + 5 + 3 if batch["node_start"][6] - batch["node_start"][5] == 3 else 0] = np.nan
    _check_tree(sv, batch, 3, 3)


def test_tree_uniforms_that_are_none_refuse(sv):
    batch = ref.random_tree_batch(16, 30, 300, 5, 3, True, "mixed", noise=0.3)
    batch["u_accept"][:] = np.nan
    w, cnt = _check_tree(sv, batch, 5, 3)
    assert cnt[1] == 0 and cnt[3] > 0


@pytest.mark.parametrize("kind,replacement", [("sampled", True), ("sampled", False), ("certain", True)])
def test_tree_keeps_the_target_law(sv, kind, replacement):
    # one place with three candidates over six tokens: the first emitted token is distributed as p
    from scipy.stats import chi2
    B, V, W = 60000, 6, 3
    g = _gen(31 + replacement)
    p1 = torch.tensor([0.32, 0.05, 0.2, 0.03, 0.3, 0.1])
    q1 = torch.tensor([0.1, 0.3, 0.25, 0.15, 0.05, 0.15])
    toks = torch.multinomial(q1.expand(B, V).cuda(), W, replacement=replacement, generator=g)
    start = (torch.arange(B + 1, device="cuda") * W).int()
    p = p1.expand(B * (W + 1), V).contiguous().cuda()
    q = q1.unsqueeze(0).contiguous().cuda()
    row = torch.full((B, W + 1), -1, dtype=torch.int32, device="cuda")
    if kind == "sampled":
        row[:, 0] = 0
    out = sv.verify_tree(p, q, toks.reshape(-1).int(), torch.full((B * W,), -1, dtype=torch.int32, device="cuda"),
                         row.reshape(-1), start, torch.rand(B * W, generator=g, device="cuda"),
                         torch.rand(B, generator=g, device="cuda"), max_nodes=W, max_depth=1, replacement=replacement)
    count = torch.bincount(out["tokens"][:, 0].long(), minlength=V).double().cpu()
    stat = float(((count - B * p1.double()) ** 2 / (B * p1.double())).sum())
    assert stat < chi2.ppf(1 - 1e-4, V - 1), stat
    assert int(out["accepted_len"].sum()) > B // 4


def test_tree_results_do_not_depend_on_the_batch(sv):
    batch = ref.random_tree_batch(21, 100, 7000, 6, 4, True, "mixed", noise=1.0)
    whole, _ = _run_tree(sv, batch, 6, 4)
    st = batch["node_start"]
    for b in (0, 17, 99):
        lo, hi = st[b], st[b + 1]
        one = dict(p=batch["p"][lo + b:hi + b + 1], q=batch["q"], tokens=batch["tokens"][lo:hi],
                   parent=batch["parent"][lo:hi], draft_row=batch["draft_row"][lo + b:hi + b + 1],
                   node_start=np.array([0, hi - lo], np.int32), u_accept=batch["u_accept"][lo:hi],
                   u_pick=batch["u_pick"][b:b + 1])
        got, _ = _run_tree(sv, one, 6, 4)
        assert np.array_equal(got["tokens"][0], whole["tokens"][b])
        assert np.array_equal(got["accept_prob"], whole["accept_prob"][lo:hi])


def test_tree_leaves_what_belongs_to_no_sequence(sv):
    batch = ref.random_tree_batch(22, 5, 300, 4, 4, True, "sampled")
    n = len(batch["tokens"])
    more = dict(batch, tokens=np.append(batch["tokens"], [5, 6]).astype(np.int32),
                parent=np.append(batch["parent"], [-1, -1]).astype(np.int32),
                u_accept=np.append(batch["u_accept"], [0.5, 0.5]).astype(np.float32),
                p=np.concatenate([batch["p"], batch["p"][:2]]),
                draft_row=np.append(batch["draft_row"], [-1, -1]).astype(np.int32))
    out = dict(accepted_len=torch.full((5,), 77, dtype=torch.int32, device="cuda"),
               tokens=torch.full((5, 5), 77, dtype=torch.int32, device="cuda"),
               path=torch.full((5, 4), 77, dtype=torch.int32, device="cuda"),
               accept_prob=torch.full((n + 2,), 77.0, device="cuda"),
               flags=torch.full((n + 2,), 77, dtype=torch.int8, device="cuda"))
    got, _ = _run_tree(sv, more, 4, 4, out=out)
    assert (got["accept_prob"][n:] == 77).all() and (got["flags"][n:] == 77).all()
    assert (got["accepted_len"] < 77).all()


def test_tree_captured_on_another_stream(sv):
    batch = ref.random_tree_batch(23, 16, 20000, 5, 5, True, "mixed", noise=1.0)
    t = ref.on_gpu(batch)
    args = [t[k] for k in ("p", "q", "tokens", "parent", "draft_row", "node_start", "u_accept", "u_pick")]
    eager = sv.verify_tree(*args, max_nodes=5, max_depth=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = sv.verify_tree(*args, max_nodes=5, max_depth=5)
        for v in out.values():
            v.fill_(55)
        graph.replay()
        again = sv.verify_tree(*args, max_nodes=5, max_depth=5)  # eager beside the captured one
    torch.cuda.synchronize()
    for k in eager:
        assert torch.equal(eager[k], out[k]) and torch.equal(eager[k], again[k])


# ------------------------------------------------------------- together

def test_chain_agrees_with_the_verifier(sv):
    """Logits through softmax and the tree call give what spec_verify_run gives for the same uniforms."""
    B, k, V = 50, 4, 257
    g = _gen(41)
    Lt = torch.randn(B, k + 1, V, generator=g, device="cuda") * 2
    Ld = (Lt[:, :k] + torch.randn(B, k, V, generator=g, device="cuda")).contiguous()
    D = torch.multinomial(torch.softmax(Ld.view(-1, V) / 0.8, 1), 1, generator=g).view(B, k).int()
    u0, u1 = torch.rand(B, k, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda")
    ver = sv.SpecVerifier(B, k, V)
    a = ver.run(Lt, Ld, D, 0.8, u_accept=u0, u_residual=u1)
    p, q = sv.softmax(Lt.view(-1, V), 0.8), sv.softmax(Ld.view(-1, V), 0.8)
    i = torch.arange(B, device="cuda", dtype=torch.int32)
    j = torch.arange(k + 1, device="cuda", dtype=torch.int32)
    row = torch.where(j[None] < k, i[:, None] * k + j[None], -1).int().reshape(-1)
    b = sv.verify_tree(p, q, D.reshape(-1), (j[:k] - 1).repeat(B), row, (torch.arange(B + 1, device="cuda") * k).int(),
                       u0.reshape(-1), u1, max_nodes=k, max_depth=k)
    r = O.verify(Lt.cpu().numpy(), Ld.cpu().numpy(), D.cpu().numpy(), 0.8, np.zeros(B, np.uint8), np.full(B, 0.5),
                 u0=u0.cpu().numpy(), u1=u1.cpu().numpy())
    clear = torch.as_tensor(r["margin"] >= 1e-6)
    assert int(clear.sum()) > 40
    assert torch.equal(a["accepted_len"].cpu()[clear], b["accepted_len"].cpu()[clear])
    assert torch.equal(a["tokens"].cpu()[clear], b["tokens"].cpu()[clear])
    f = b["flags"].view(B, k)
    assert torch.equal(a["flags"].cpu()[clear], f.cpu()[clear])
    tested = (f != 0) & clear.cuda()[:, None]
    torch.testing.assert_close(a["accept_prob"][tested], b["accept_prob"].view(B, k)[tested], rtol=2e-5, atol=0)
    ver.close()


def test_hidden_states_to_accepted_tokens(sv):
    """Draft blocks, output heads, probabilities and a tree, one after another, against 64 bits at each step."""
    B, G, H, V = 6, 3, 256, 2000
    g = _gen(51)
    hidden = torch.randn(B, H, generator=g, device="cuda").to(torch.bfloat16)
    w_block = (torch.randn(G, H, H, generator=g, device="cuda") / 16).to(torch.bfloat16)
    head = (torch.randn(V, H, generator=g, device="cuda") / 5).to(torch.bfloat16)
    blocks = torch.empty(B, G, H, dtype=torch.bfloat16, device="cuda")
    sv.linear(hidden, w_block, residual=hidden.unsqueeze(0).expand(G, B, H), activation="silu",
              out=blocks.transpose(0, 1))
    ref.assert_linear(blocks.transpose(0, 1), hidden, w_block, None, hidden.unsqueeze(0).expand(G, B, H), "silu", 0)
    draft_logits = sv.linear(blocks.view(B * G, H), head, activation="softcap", cap=20.0, out_dtype=torch.float32)
    ref.assert_linear(draft_logits, blocks.view(B * G, H), head, None, None, "softcap", 20.0)
    q = sv.softmax(draft_logits, 0.9)
    _assert_softmax(q, draft_logits, 0.9)
    # two candidates for the first place, chains of the further heads behind the first one
    two = torch.multinomial(q.view(B, G, V)[:, 0], 2, replacement=True, generator=g)
    more = torch.multinomial(q, 1, generator=g).view(B, G)[:, 1:]
    tokens = torch.cat([two, more], 1).int()
    parent = torch.tensor([-1, -1, 0, 2], dtype=torch.int32, device="cuda").repeat(B)
    n = 4
    target_hidden = torch.randn(B * (n + 1), H, generator=g, device="cuda") * 0.3
    target_hidden = (target_hidden + hidden.repeat_interleave(n + 1, 0)).to(torch.bfloat16)
    target_logits = sv.linear(target_hidden, head, activation="softcap", cap=20.0, out_dtype=torch.float32)
    p = sv.softmax(target_logits, 0.9)
    base = torch.arange(B, device="cuda", dtype=torch.int32)[:, None] * G
    row = torch.cat([base, base + 1, torch.full_like(base, -1), base + 2, torch.full_like(base, -1)], 1).reshape(-1)
    batch = dict(p=p, q=q, tokens=tokens.reshape(-1), parent=parent, draft_row=row.int(),
                 node_start=(torch.arange(B + 1, device="cuda") * n).int(),
                 u_accept=torch.rand(B * n, generator=g, device="cuda"), u_pick=torch.rand(B, generator=g, device="cuda"))
    batch = {k: v.contiguous().cpu().numpy() for k, v in batch.items()}
    _check_tree(sv, batch, n, 3)


@pytest.mark.parametrize("per_position", [False, True])
def test_run_hidden_is_the_heads_and_the_verifier(sv, per_position):
    B, k, H, V = 9, 3, 128, 3000
    g = _gen(61 + per_position)
    th = torch.randn(B, k + 1, H, generator=g, device="cuda").to(torch.bfloat16)
    dh = torch.randn(B, k, 64, generator=g, device="cuda").to(torch.bfloat16)
    wt = (torch.randn(V, H, generator=g, device="cuda") / 4).to(torch.bfloat16)
    shape = (k, V, 64) if per_position else (V, 64)
    wd = (torch.randn(shape, generator=g, device="cuda") / 4).to(torch.bfloat16)
    bias = torch.randn(shape[:-1], generator=g, device="cuda")
    D = torch.randint(0, V, (B, k), generator=g, device="cuda").int()
    ver = sv.SpecVerifier(B, k, V)
    out = ver.run_hidden(th, wt, dh, wd, D, 0.9, draft_bias=bias, cap=15.0, seed=5, logits_dtype=torch.float32)
    ref.assert_linear(out["target_logits"].view(-1, V), th.view(-1, H), wt, None, None, "softcap", 15.0)
    if per_position:
        ref.assert_linear(out["draft_logits"].transpose(0, 1), dh.transpose(0, 1), wd, bias, None, "softcap", 15.0)
    else:
        ref.assert_linear(out["draft_logits"].view(-1, V), dh.view(-1, 64), wd, bias, None, "softcap", 15.0)
    same = ver.run(out["target_logits"], out["draft_logits"], D, 0.9, seed=5)
    for name in ("accepted_len", "tokens", "accept_prob", "flags"):
        assert torch.equal(out[name], same[name])
    ver.close()


# ------------------------------------------------------------- results on a stream of their own

def test_results_belong_to_the_stream_of_the_call(sv):
    """With ``stream=`` a new result is never memory that the current stream may still use, nor is a dropped one given
    to the current stream, in whose order the call does not stand."""
    g = _gen(71)
    B, k, H, V = 5, 2, 64, 300000
    x = torch.randn(B, H, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(V, H, generator=g, device="cuda") / 8).to(torch.bfloat16)
    th, dh = x.unsqueeze(1).repeat(1, k + 1, 1), x.unsqueeze(1).repeat(1, k, 1)
    D = torch.randint(0, V, (B, k), generator=g, device="cuda").int()
    logits = sv.linear(x, w, out_dtype=torch.float32)
    probs = sv.softmax(logits, 0.9)
    i32 = dict(dtype=torch.int32, device="cuda")
    nodes = 4
    tree = (probs[:nodes + 1], probs[:1], torch.tensor([1, 2, 3, 4], **i32), torch.full((nodes,), -1, **i32),
            torch.tensor([0, -1, -1, -1, -1], **i32), torch.tensor([0, nodes], **i32), torch.rand(nodes, generator=g, device="cuda"),
            torch.rand(1, generator=g, device="cuda"))
    Lt, Ld = logits.unsqueeze(1).repeat(1, k + 1, 1), logits.unsqueeze(1).repeat(1, k, 1)
    ver = sv.SpecVerifier(B, k, V)

    def places(tensors):
        return [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in tensors]

    def meet(a, b):
        return any(x[0] < y[1] and y[0] < x[1] for x in a for y in b)

    calls = [lambda s: dict(y=sv.linear(x, w, out_dtype=torch.float32, stream=s)),
             lambda s: dict(y=sv.softmax(logits, 0.9, stream=s)),
             lambda s: sv.verify_tree(*tree, max_nodes=nodes, max_depth=nodes, stream=s),
             lambda s: ver.run_hidden(th, w, dh, w, D, 0.9, seed=3, logits_dtype=torch.float32, stream=s),
             lambda s: ver.run(Lt, Ld, D, 0.9, seed=3, row_stats=True, stream=s)]
    for call in calls:
        want = {n: v.clone() for n, v in call(None).items()}
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        for handle in (side.cuda_stream, side):
            # blocks of every result's size that the current stream has used and given back
            freed = [torch.empty_like(v) for v in want.values() for _ in range(3)]
            ours = places(freed)
            del freed
            got = call(handle)
            theirs = places(got.values())
            assert not meet(ours, theirs)
            side.synchronize()
            for n in want:
                assert torch.equal(got[n], want[n]), n
            del got
            again = [torch.empty_like(v) for v in want.values() for _ in range(3)]
            assert not meet(theirs, places(again))
            del again
        # the current stream by its handle, the default stream among them
        got = call(torch.cuda.current_stream().cuda_stream)
        with torch.cuda.stream(side):
            far = call(torch.cuda.default_stream().cuda_stream)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]) and torch.equal(far[n], want[n]), n
    ver.close()


@pytest.mark.parametrize("M,odd", [(1, 0), (3, 1), (130, 0)])
@pytest.mark.parametrize("K", [65600, 1 << 20])
def test_linear_bf16_results_of_very_long_sums(sv, M, odd, K):
    # Sums of one sign.  Each step of 16 products cuts off up to 2^-23 of the sum so far for each of them and the sum
    # itself; a sum grows evenly, so n steps are short of up to 17 n 2^-24 of it.  At most 2048 steps go into one sum, and
    # the additions of the K / 512 segments' sums are off by half a step each; then comes the rounding to bf16, up to 2^-8.
    g, N = _gen(M + K), 400
    x = torch.rand(M, K + odd, generator=g, device="cuda").to(torch.bfloat16)[:, odd:]
    w = torch.rand(N, K + odd, generator=g, device="cuda")
    w = (w * torch.linspace(1, 2, N, device="cuda").unsqueeze(1)).to(torch.bfloat16)[:, odd:]
    want = torch.cat([x.double() @ part.double().T for part in w.split(50)], 1)
    off = (sv.linear(x, w).double() - want) / want
    own = 17 * 2048 * 2.0 ** -24 + K / 512 * 2.0 ** -24
    assert float(off.abs().max()) <= 2.0 ** -8 * (1 + own) + own
    # the sums lie evenly over a binade, so their roundings have no side: within 4 deviations of a mean over N of them
    assert abs(float(off.mean())) <= own + 4 * 2.0 ** -8 / 3 ** 0.5 / N ** 0.5, float(off.mean())


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_sums_that_take_seconds(sv, dtype, odd):
    # a wait gives up after two seconds without an answer, not where a tile takes that long: all ones, so every sum of 512
    # is exact, and so are the sums of these up to 2^33 (24 bits above 2^9); the last one is a single entry
    K = (1 << 29) + 1
    x = torch.ones(K + odd, dtype=torch.bfloat16, device="cuda")[odd:].unsqueeze(0)
    y = sv.linear(x, x, out_dtype=dtype)
    assert float(y) == float(torch.tensor(float(K)).to(dtype))


def _by_bias(sv, z, act, cap=1.0, dtype=torch.float32, M=1):
    """An activation of z itself: without entries of K its argument is the bias."""
    empty = torch.empty(M, 0, dtype=torch.bfloat16, device="cuda")
    return sv.linear(empty, torch.empty(len(z), 0, dtype=torch.bfloat16, device="cuda"), bias=z, activation=act, cap=cap,
                     out_dtype=dtype)[0]


@pytest.mark.parametrize("cap", [2.0 ** -128 * (1 + 2.0 ** -20), 5e-39, 1.2e-38, 1e-30, 1.0, 5.0, 1e30, 1e38, 3.4028234663852886e38])
def test_linear_soft_cap_of_any_size(sv, cap):
    # tanh's argument is off by 2 half steps and, of caps above 2^126, by 4 more (2^-22, as their reciprocals have fewer
    # digits); tanh by 4 more, the product by 1; results below the normal floats by a step of those
    cap = float(torch.tensor(cap))  # as an fp32 number has it
    z = torch.cat([torch.tensor([0.0, -0.0, float("inf"), -float("inf")]), torch.logspace(-44.8, 38.5, 4000),
                   -torch.logspace(-44.8, 38.5, 4000)])
    near = torch.tensor(cap, dtype=torch.float64) * torch.logspace(-6, 2, 2000, dtype=torch.float64)
    z = torch.cat([z, near.clamp(max=3.4e38).float(), -near.clamp(max=3.4e38).float()]).cuda()
    got, want = _by_bias(sv, z, "softcap", cap).double(), ref.ACT["softcap"](z.double(), cap)
    steps = 11 if cap > 2.0 ** 126 else 8
    off = (got - want).abs()
    bound = steps * 2.0 ** -24 * want.abs() + 2.0 ** -149
    assert bool((off <= bound).all()), (float(z[(off / bound).argmax()]), float((off / bound).max()))
    # a bf16 result: a rounding more.  The largest bf16 number is (2 - 2^-7) 2^127; what is nearer to 2^128 is infinite.
    short = _by_bias(sv, z, "softcap", cap, torch.bfloat16).double()
    there = want.abs() < (2 - 2.0 ** -8) * 2.0 ** 127 * (1 - 12 * 2.0 ** -24)
    assert bool(((short - want).abs() <= (2.0 ** -8 + 12 * 2.0 ** -24) * want.abs() + 2.0 ** -133)[there].all())
    assert torch.equal(short[~there].abs(), torch.full_like(short[~there], float("inf")))


@pytest.mark.parametrize("V,n", [(8, 4), (20, 7), (600, 12), (5000, 9)])
def test_tree_siblings_offered_twice_without_replacement(sv, V, n):
    """A sibling that was offered before has no place in what is left of the proposal: its mu is 0, and its mass is
    taken out once.  Against the distributions themselves, candidate by candidate."""
    B = 60
    rng = np.random.default_rng(V)
    logits = rng.standard_normal((B, V))
    p = np.zeros((B * (n + 1), V), np.float32)
    p[::n + 1] = ref._softmax(2 * logits)
    p[p.sum(1) == 0] = 1.0 / V
    q = ref._softmax(2 * logits + 1.5 * rng.standard_normal((B, V))).astype(np.float32)
    few = [rng.choice(V, 1 + n // 2, replace=False, p=r / r.sum()) for r in q.astype(np.float64)]
    tokens = np.stack([rng.choice(f, n) for f in few]).astype(np.int32)  # n places, half as many tokens
    u, u_pick = rng.random((B, n)).astype(np.float32) * 0.999, rng.random(B).astype(np.float32) * 0.999
    row = np.full((B, n + 1), -1, np.int32)
    row[:, 0] = np.arange(B)
    alpha, flags, tok = np.zeros((B, n)), np.zeros((B, n), np.int8), np.full((B, 2), -1, np.int32)
    twice = 0
    for b in range(B):
        rest, prop, seen = p[b * (n + 1)].astype(np.float64), q[b].astype(np.float64), []
        Z = 1.0
        for i in range(n):
            v = tokens[b, i]
            twice += v in seen
            mu = prop / (1.0 - prop[seen].sum())
            mu[seen] = 0.0
            alpha[b, i] = min(1.0, rest[v] / (Z * mu[v])) if mu[v] > 0 else float(rest[v] > 0)
            if rest[v] > 0 and u[b, i] * mu[v] * Z <= rest[v]:
                flags[b, i], tok[b] = ref.ACCEPT, (v, 0)
                break
            flags[b, i] = ref.REJECT
            rest = np.maximum(rest / Z - mu, 0.0)
            Z = rest.sum()
            if v not in seen:
                seen.append(v)
        if flags[b].max() == ref.REJECT and not (flags[b] == ref.ACCEPT).any():
            tok[b, 0] = ref.pick(rest if Z > 0 else p[b * (n + 1)].astype(np.float64), u_pick[b])
        else:
            tok[b, 1] = ref.pick(p[b * (n + 1) + 1 + int(np.argmax(flags[b] == ref.ACCEPT))].astype(np.float64), u_pick[b])
    assert twice > B // 4
    batch = dict(p=p, q=q, tokens=tokens.reshape(-1), parent=np.full(B * n, -1, np.int32), draft_row=row.reshape(-1),
                 node_start=(np.arange(B + 1) * n).astype(np.int32), u_accept=u.reshape(-1), u_pick=u_pick)
    got, _ = _run_tree(sv, batch, n, 1, False)
    assert np.array_equal(got["flags"].reshape(B, n), flags)
    np.testing.assert_allclose(got["accept_prob"].reshape(B, n), alpha, rtol=2.0 ** -24 + 1e-9, atol=1e-30)
    assert np.array_equal(got["tokens"], tok)


@pytest.mark.parametrize("spread", [0.3, 1.0])
def test_linear_fp32_gelu_is_as_good_as_its_roundings(sv, spread):
    # The argument's rounding, the sum's and the product's two are even, of a third of a squared half step at most each,
    # and erff's own error is taken for a fifth: sqrt(5 / 3) half steps in the 2-norm.
    z = torch.randn(1000000, generator=_gen(81), device="cuda") * spread
    got, want = _by_bias(sv, z, "gelu").double(), ref.ACT["gelu"](z.double(), 1.0)
    assert float((got - want).norm() / want.norm()) <= (5 / 3) ** 0.5 * 2.0 ** -24


def test_linear_as_many_groups_as_memory_holds(sv):
    # 2^28 groups of eight odd rows: in classes of rows that start alike they would be 2^31 tiles
    G, N, K = 1 << 28, 8, 3
    g = _gen(91)
    x = torch.randn(1, K, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(1, N, K, generator=g, device="cuda").to(torch.bfloat16)
    y = sv.linear(x, w.expand(G, N, K))
    ref.assert_linear(y[0], x, w[0], None, None, "none", 0.0)
    assert bool((y == y[0]).all())


# ------------------------------------------------------------- the ends of the documented ranges

def _far_rows(seed, rows, V, dtype, odd):
    """Logits rows; `odd`: at odd addresses, NaN between them."""
    g = _gen(seed)
    if not odd:
        return (torch.randn(rows, V, generator=g, device="cuda") * 4).to(dtype)
    store = torch.full((1 + rows * (V + 3),), float("nan"), dtype=dtype, device="cuda")
    x = store[1:].view(rows, V + 3)[:, :V]
    x.copy_(torch.randn(rows, V, generator=g, device="cuda") * 4)
    return x


# a row in registers, clusters of sixteen that take several rows, rows longer than the registers of sixteen CTAs
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,odd", [(40, 140000, False), (40, 151936, True), (3, 262144, False), (3, 262145, False),
                                        (2, 300001, True), (20, 300000, False), (3, 1 << 22, False), (2, (1 << 22) - 1, True)])
def test_softmax_long_rows(sv, dtype, rows, V, odd):
    x = _far_rows(rows + V, rows, V, dtype, odd)
    t = torch.rand(rows, generator=_gen(V), device="cuda") + 0.3
    t[rows // 2] = 0.0
    out = torch.full((rows, V + 2), 9.0, device="cuda")
    y = sv.softmax(x, t, out=out[:, 1:V + 1])
    warm = t > 0
    _assert_softmax(y[warm], x[warm], t[warm])
    cold = x[rows // 2].float()
    assert torch.equal(y[rows // 2], torch.nn.functional.one_hot(cold.argmax(), V).float())
    assert bool((out[:, 0] == 9).all()) and bool((out[:, -1] == 9).all())


@pytest.mark.parametrize("V", [262145, 300001, 1 << 22])
def test_softmax_long_rows_in_place(sv, V):
    x = _far_rows(V, 4, V, torch.float32, False)
    x[2, V - 3] = x[2, 70000] = 60.0
    before, t = x.clone(), torch.tensor([0.7, 1.3, 0.0, 1e-30], device="cuda")
    sv.softmax(x, t, out=x)
    _assert_softmax(x[:2], before[:2], t[:2])
    want = torch.zeros_like(x[2:])
    want[0, 70000] = 1
    want[1, before[3].argmax()] = 1
    assert torch.equal(x[2:], want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [262145, 1 << 22])
def test_softmax_long_rows_without_a_distribution(sv, dtype, V):
    x = _far_rows(V, 9, V, dtype, False)
    x[1, V - 1] = float("nan")
    x[2, V // 2] = float("inf")
    x[3] = float("-inf")
    x[4, : V - 1] = float("-inf")
    x[5] = torch.finfo(dtype).min
    t = torch.ones(9, device="cuda")
    t[6], t[7], t[8] = -1.0, float("nan"), float("inf")
    y = sv.softmax(x, t)
    assert bool(torch.isnan(y[[1, 2, 3, 6, 7, 8]]).all())
    assert float(y[4, V - 1]) == 1.0 and float(y[4].sum()) == 1.0
    _assert_softmax(y[[0, 5]], x[[0, 5]], 1.0)
    cold = sv.softmax(x, torch.where(t > 0, 0.0, t))
    assert bool(torch.isnan(cold[[1, 2, 3, 6, 7]]).all())
    assert torch.equal(cold[[0, 4, 5]].argmax(1), x[[0, 4, 5]].float().argmax(1))
    assert bool((cold[[0, 4, 5]].sum(1) == 1).all())


@pytest.mark.parametrize("V,kind", [(300001, "mixed"), (1 << 22, "sampled"), ((1 << 22) - 1, "certain")])
def test_tree_the_longest_rows(sv, V, kind):
    batch = ref.random_tree_batch(V, 2, V, 4, 3, True, kind, sharp=3.0, noise=1.0)
    _check_tree(sv, batch, 4, 3)


@pytest.mark.parametrize("V", [2200001, 1 << 22])
def test_tree_one_cta_for_the_longest_rows(sv, V):
    # so many sequences that each has one CTA, with more than 4096 sums of a row; all share one row of each side
    B = 170
    rng = np.random.default_rng(V)
    logits = rng.standard_normal(V, dtype=np.float32) * 2
    p = ref._softmax(logits[None].astype(np.float64)).astype(np.float32)
    q = ref._softmax((logits + 0.4 * rng.standard_normal(V, dtype=np.float32))[None].astype(np.float64)).astype(np.float32)
    sums = np.cumsum(q[0].astype(np.float64))
    tokens = np.searchsorted(sums, rng.random(B) * sums[-1], side="right").clip(max=V - 1).astype(np.int32)
    row = np.stack([np.zeros(B), np.full(B, -1)], 1).astype(np.int32).reshape(-1)
    batch = dict(tokens=tokens, parent=np.full(B, -1, np.int32), draft_row=row, node_start=np.arange(B + 1, dtype=np.int32),
                 u_accept=rng.random(B).astype(np.float32), u_pick=np.minimum(rng.random(B), 1 - 2.0 ** -24).astype(np.float32))
    t = {k: torch.as_tensor(v).cuda() for k, v in batch.items()}
    cnt = torch.zeros(8, dtype=torch.int64, device="cuda")
    out = sv.verify_tree(torch.as_tensor(p).cuda().expand(2 * B, V), torch.as_tensor(q).cuda(), t["tokens"], t["parent"],
                         t["draft_row"], t["node_start"], t["u_accept"], t["u_pick"], max_nodes=1, max_depth=1, counters=cnt)
    # the tokens of either row by its sums, in 64 bits
    p64, q64 = p[0].astype(np.float64), q[0].astype(np.float64)
    alpha = np.minimum(1.0, p64[tokens] / q64[tokens])
    yes = batch["u_accept"].astype(np.float64) * q64[tokens] <= p64[tokens]
    rest_sums, p_sums = np.cumsum(np.maximum(p64 - q64, 0.0)), np.cumsum(p64)
    u = batch["u_pick"].astype(np.float64)
    assert 5 < (~yes).sum() < B - 5
    pick = np.where(yes, np.searchsorted(p_sums, u * p_sums[-1], side="right"),
                    np.searchsorted(rest_sums, u * rest_sums[-1], side="right"))
    want = dict(accepted_len=yes.astype(np.int32), path=np.where(yes, 0, -1).astype(np.int32)[:, None],
                tokens=np.stack([np.where(yes, tokens, pick), np.where(yes, pick, -1)], 1).astype(np.int32),
                flags=np.where(yes, ref.ACCEPT, ref.REJECT).astype(np.int8), accept_prob=alpha)
    counts = np.array([B, yes.sum(), 0, (~yes).sum(), yes.sum(), 0, 0, 0])
    _assert_tree(({k: v.cpu().numpy() for k, v in out.items()}, cnt.cpu().numpy()), (want, counts))


def test_calls_that_would_write_over_their_inputs_are_refused(sv):
    g = _gen(95)
    h = torch.randn(6, 256, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(256, 256, generator=g, device="cuda") / 16).to(torch.bfloat16)
    before = h.clone()
    shared = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    f32 = torch.zeros(6, 256, device="cuda")
    for kw in (dict(x=h, residual=h, out=h), dict(x=h, out=h), dict(x=h, out=w[:6]), dict(x=h, out=w[100:106]),
               dict(x=shared[:1536].view(6, 256), out=shared[768:2304].view(6, 256)),
               dict(x=h, bias=f32[2], out=f32), dict(x=h, residual=f32[:1].expand(6, 256), out=f32),
               dict(x=h, residual=f32.view(torch.bfloat16)[:3].view(6, 256), out=f32)):
        with pytest.raises(sv.SpecVerifyError):
            sv.linear(kw.pop("x"), w, **kw)
    for logits, out in ((f32, f32.view(-1)[:1530].view(6, 255)), (f32.view(torch.bfloat16)[:3].view(6, 256), f32),
                        (f32.view(-1)[256:].view(5, 256), f32[:5])):
        with pytest.raises((sv.SpecVerifyError, ValueError)):
            sv.softmax(logits, 1.0, out=out)
    assert torch.equal(h, before)
    # rows that lie between another operand's rows, and neighbours, are taken
    both = torch.zeros(6, 512, dtype=torch.bfloat16, device="cuda")
    both[:, :256] = h
    sv.linear(both[:, :256], w, residual=both[:, :256], out=both[:, 256:])
    ref.assert_linear(both[:, 256:], h, w, None, h, "none", 0.0)
    rows = torch.zeros(12, 256, dtype=torch.bfloat16, device="cuda")
    rows[6:] = h
    sv.linear(rows[6:], w, out=rows[:6])
    ref.assert_linear(rows[:6], h, w, None, None, "none", 0.0)
    wide = torch.randn(6, 300, generator=g, device="cuda")
    p = sv.softmax(wide[:, :100], 1.0, out=wide[:, 100:200])
    _assert_softmax(p, wide[:, :100], 1.0)
