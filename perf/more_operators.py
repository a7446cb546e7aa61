"""Cases of the operators around a tree's target pass: penalties, biases and masks on logits rows, the cache in
pages of 8-bit entries (rows written, accepted rows kept) and the attention of drafted trees over it.

``run`` computes them with elementary torch operations where ``own`` is false
and through the package's entry points where it is true.
"""
import math

import torch

own = False

MAX_CACHE = 1.1e9  # bytes of keys and values that the largest attention drawn reads
MAX_FLOPS = 1.2e11


def listed():
    return [
        # one sequence's chain of four drafts in front of the verifying call, a short history
        dict(name="penalties_b1_v32000", op="penalties", b=1, widths="1,1,1,1", v=32000, dtype="f32", out="same", cap=256,
             ragged=False, repetition=False, biases=0, masks=False),
        # the 128K-vocabulary batch, in place: only tokens of the histories change
        dict(name="penalties_b64_v128256", op="penalties", b=64, widths="1,1,1,1,1", v=128256, dtype="bf16", out="same",
             cap=4096, ragged=True, repetition=False, biases=0, masks=False),
        # trees under a grammar, a mask for each node, biases, all penalties, logits kept
        dict(name="penalties_tree_b32_v151936", op="penalties", b=32, widths="3,2,2", v=151936, dtype="bf16", out="f32",
             cap=1000, ragged=True, repetition=True, biases=300, masks=True),
        # the rows of one sequence's chain of four drafts
        dict(name="write_b1", op="write", b=1, widths="1,1,1,1", rows=0, heads=8, dim=128, page=64, block=16, context=500,
             dtype="bf16"),
        # of a batch of trees with 21 nodes each
        dict(name="write_tree_b64", op="write", b=64, widths="3,2,2", rows=0, heads=8, dim=128, page=64, block=32,
             context=1000, dtype="bf16"),
        # prompts of up to 2048 tokens into empty pages
        dict(name="write_prompts_b32", op="write", b=32, widths="", rows=2048, heads=8, dim=128, page=64, block=64,
             context=0, dtype="bf16"),
        # the accepted drafts of one sequence in the sixteen layers of a small model
        dict(name="keep_b1_l16", op="keep", b=1, widths="1,1,1,1", layers=16, heads=8, dim=64, page=64, block=16,
             context=200),
        # the accepted paths of 64 trees in 16 layers
        dict(name="keep_b64_l16", op="keep", b=64, widths="3,2,2", layers=16, heads=8, dim=128, page=64, block=32,
             context=130),
        # plain decoding of one sequence
        dict(name="attend_b1_c1000", op="attend", b=1, widths="", context=1000, heads=8, group=4, dim=128, page=64,
             block=64, ragged=False),
        # a batch of chains over contexts of up to 8192 tokens
        dict(name="attend_b64_c8192", op="attend", b=64, widths="1,1,1,1,1", context=8192, heads=8, group=4, dim=128,
             page=64, block=64, ragged=True),
        # trees of 21 nodes, eight query heads to a key head, small pages and blocks
        dict(name="attend_tree_b32_c4000", op="attend", b=32, widths="3,2,2", context=4000, heads=4, group=8, dim=128,
             page=16, block=16, ragged=True),
        # two long contexts of an odd length, heads of 64
        dict(name="attend_b2_c131071", op="attend", b=2, widths="1,1,1,1", context=131071, heads=8, group=5, dim=64,
             page=128, block=64, ragged=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


TREES = ["", "1", "1,1,1", "1,1,1,1,1,1,1,1", "4", "2,2,2", "4,2,1,1", "8,1"]


def draw(rng):
    op = rng.choice(["penalties", "write", "keep", "attend", "attend"])
    widths = rng.choice(TREES)
    nodes = len(_parents(widths)[0])
    if op == "penalties":
        v = _spread(rng, 1000, 262144)
        masks = rng.random() < 0.5
        return dict(op=op, b=max(1, min(_spread(rng, 1, 256), int(8e7 / (v * (nodes + 1))))), widths=widths, v=v,
                    dtype=rng.choice(["bf16", "f32"]), out=rng.choice(["same", "f32", "bf16"]),
                    cap=_spread(rng, 1, 32768), ragged=rng.random() < 0.7, repetition=rng.random() < 0.5,
                    biases=rng.choice([0, 0, _spread(rng, 1, 300)]), masks=masks)
    heads, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    block = rng.choice([s for s in (8, 16, 32, 64, 128) if s <= page])
    if op == "write":
        rows = _spread(rng, 2, 4096) if rng.random() < 0.5 else 0
        b = _spread(rng, 1, 256)
        if rows:
            b = max(1, min(b, int(6.5e7 / (rows * heads * dim))))
        return dict(op=op, b=b, widths="" if rows else widths, rows=rows, heads=heads, dim=dim, page=page, block=block,
                    context=rng.choice([0, _spread(rng, 1, 1000)]), dtype=rng.choice(["bf16", "f32"]))
    if op == "keep":
        b, context = _spread(rng, 1, 128), _spread(rng, 1, 200)
        pages = (context + nodes + page) // page + 1
        layers = max(1, min(rng.choice([1, 4, 16, 32]), int(2.5e8 / (b * pages * page * heads * dim))))
        return dict(op=op, b=b, widths=widths or "1", layers=layers, heads=heads, dim=dim, page=page, block=block,
                    context=context)
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    context = _spread(rng, 1, 131072)
    most = min(MAX_CACHE / (2.0 * heads * dim * (context + 300)),
               MAX_FLOPS / (4.0 * (nodes + 1) * heads * group * dim * (context + 300)))
    return dict(op=op, b=max(1, min(_spread(rng, 1, 256), int(most))), widths=widths, context=context, heads=heads,
                group=group, dim=dim, page=page, block=block, ragged=rng.random() < 0.5)


def _parents(widths):
    """Parent of each node of the full tree, level by level (-1: the root), and the node's depth."""
    parent, depth, last = [], [], [-1]
    for at, w in enumerate(int(w) for w in widths.split(",") if w):
        level = []
        for node in last:
            for _ in range(w):
                level.append(len(parent))
                parent.append(node)
                depth.append(at)
        last = level
    return parent, depth


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _lengths(n, ragged, b, g):
    """b lengths of up to n: the same ones for every seed, in another order."""
    full = torch.full((b,), n, device="cuda")
    if not ragged:
        return full
    low = (n + 1) // 2
    steps = torch.randperm(b, generator=g, device="cuda")
    return low + (steps * (n - low) // max(1, b - 1) if b > 1 else torch.zeros_like(steps))


def _tree(case, g, ragged):
    """Nodes of b trees: parent, tokens' count and where each sequence's nodes start."""
    parent1, depth1 = _parents(case["widths"])
    N, b = len(parent1), case["b"]
    n = _lengths(N, ragged, b, g)
    start = torch.zeros(b + 1, dtype=torch.int64, device="cuda")
    start[1:] = n.cumsum(0)
    total = int(start[-1])
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), n)
    at = torch.arange(total, device="cuda") - start[seq]
    parent = torch.tensor(parent1, dtype=torch.int64, device="cuda")[at]
    return dict(parent=parent.to(torch.int32), node_start=start.to(torch.int32), total=total, max_nodes=N,
                depth=max(depth1, default=-1) + 1)


def prepare(case, seed):
    g = _generator(seed)
    return dict(penalties=_prepare_penalties, write=_prepare_write, keep=_prepare_keep, attend=_prepare_attend)[case["op"]](
        case, g)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _zipf(shape, v, g):
    """Tokens as texts repeat them: of rank 1 / u, spread over the vocabulary."""
    u = torch.rand(shape, generator=g, device="cuda")
    return (((v ** u) - 1.0).long().clamp(0, v - 1) * 7919 % v).to(torch.int32)


def _prepare_penalties(case, g):
    b, v = case["b"], case["v"]
    s = dict(case=case, **_tree(case, g, case["ragged"]))
    rows = s["total"] + b
    s["logits"] = (torch.randn(rows, v, generator=g, device="cuda") * 3.0).to(_dtype(case["dtype"]))
    s["history"] = _zipf((b, case["cap"]), v, g)
    s["history_len"] = _lengths(case["cap"], case["ragged"], b, g).to(torch.int32)
    s["prompt_len"] = s["history_len"] // 2
    s["tokens"] = _zipf((s["total"],), v, g)
    s["frequency"] = 0.2 * torch.rand(b, generator=g, device="cuda")
    s["presence"] = 0.5 * torch.rand(b, generator=g, device="cuda")
    s["repetition"] = 1.0 + 0.3 * torch.rand(b, generator=g, device="cuda") if case["repetition"] else None
    s["bias"] = None
    if case["biases"]:
        n, c = b * case["biases"], case["biases"]
        s["bias"] = (torch.arange(0, n + 1, c, dtype=torch.int32, device="cuda"),
                     torch.randint(0, v, (n,), generator=g, device="cuda").to(torch.int32),
                     torch.randn(n, generator=g, device="cuda") * 4.0)
    s["mask"] = s["mask_row"] = None
    if case["masks"]:
        # a grammar allows a few tokens, a string's inside nearly all of them; some rows have none
        words = (v + 31) // 32
        allow = torch.tensor([0.001, 0.05, 0.98], device="cuda")[torch.randint(0, 3, (rows, 1), generator=g, device="cuda")]
        s["mask"] = torch.empty(rows, words, dtype=torch.int32, device="cuda")
        step = max(1, int(2e8 / (words * 32)))
        bit = torch.arange(32, device="cuda")
        for lo in range(0, rows, step):
            part = allow[lo:lo + step, :, None]
            bits = torch.rand(part.shape[0], words, 32, generator=g, device="cuda") < part
            word = (bits.long() << bit).sum(2)
            s["mask"][lo:lo + step] = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
        at = torch.arange(rows, device="cuda")
        s["mask_row"] = torch.where(at % 7 == 3, -1, at).to(torch.int32)
    s["out"] = s["logits"] if case["out"] == "same" else torch.empty(rows, v, dtype=_dtype(case["out"]), device="cuda")
    return s


def _prepare_cache(case, g, lengths, layers=None):
    """Pages for `lengths` tokens of each sequence in any order, entries and scales as a cache in use holds them."""
    b, heads, dim, page, block = (case[f] for f in ("b", "heads", "dim", "page", "block"))
    cols = int((lengths.max() + page - 1) // page)
    pages = b * cols + 1
    lead = () if layers is None else (layers,)
    shape, scales = lead + (pages, heads, page, dim), lead + (pages, heads, page // block)

    def entries():
        out = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        flat = out.view(-1)
        step = 1 << 28
        for lo in range(0, flat.numel(), step):
            x = torch.randn(min(step, flat.numel() - lo), generator=g, device="cuda") * 90.0
            flat[lo:lo + step] = x.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        return out

    def powers():
        return 2.0 ** torch.randint(-8, -5, scales, generator=g, device="cuda")

    table = torch.randperm(pages - 1, generator=g, device="cuda")[:b * cols].view(b, cols).to(torch.int32)
    return dict(cache=(entries(), entries(), powers(), powers()), table=table)


def _prepare_write(case, g):
    b = case["b"]
    if case["rows"]:
        n = _lengths(case["rows"], True, b, g) - 1
        start = torch.zeros(b + 1, dtype=torch.int64, device="cuda")
        start[1:] = n.cumsum(0)
        s = dict(case=case, node_start=start.to(torch.int32), total=int(start[-1]), max_nodes=case["rows"] - 1)
    else:
        s = dict(case=case, **_tree(case, g, False))
    context = _lengths(case["context"], True, b, g)
    s["context"] = context.to(torch.int32)
    s.update(_prepare_cache(case, g, context + s["max_nodes"] + 1))
    shape = (s["total"] + b, case["heads"], case["dim"])
    s["k"], s["v"] = ((torch.randn(shape, generator=g, device="cuda") * 1.5).to(_dtype(case["dtype"])) for _ in range(2))
    return s


def _prepare_keep(case, g):
    b = case["b"]
    s = dict(case=case, **_tree(case, g, False))
    context = _lengths(case["context"], True, b, g)
    s["context"] = context.to(torch.int32)
    s.update(_prepare_cache(case, g, context + s["max_nodes"] + 1, case["layers"]))
    # a walk down each tree, children by chance, stopped by chance
    parent1, depth1 = _parents(case["widths"])
    parent, depth = (torch.tensor(a, device="cuda") for a in (parent1, depth1))
    path = torch.full((b, s["depth"]), -1, dtype=torch.int64, device="cuda")
    length = torch.randint(0, s["depth"] + 1, (b,), generator=g, device="cuda")
    cur = torch.full((b,), -1, dtype=torch.int64, device="cuda")
    for t in range(s["depth"]):
        luck = torch.rand(b, len(parent1), generator=g, device="cuda")
        child = torch.where((parent == cur.unsqueeze(1)) & (depth == t), luck, -1.0).argmax(1)
        cur = torch.where(length > t, child, cur)
        path[:, t] = torch.where(length > t, child, -1)
    s["path"], s["accepted_len"] = path.to(torch.int32), length.to(torch.int32)
    return s


def _prepare_attend(case, g):
    b, dim = case["b"], case["dim"]
    s = dict(case=case, **_tree(case, g, case["ragged"]))
    context = _lengths(case["context"], case["ragged"], b, g)
    s["context"] = context.to(torch.int32)
    s.update(_prepare_cache(case, g, context + s["max_nodes"] + 1))
    s["scale"] = 1.0 / math.sqrt(dim)
    rows, heads = s["total"] + b, case["heads"] * case["group"]
    s["q"] = (torch.randn(rows, heads, dim, generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    s["out"] = torch.empty_like(s["q"])
    return s


def run(s):
    op = s["case"]["op"]
    if own:
        return dict(penalties=_penalties_own, write=_write_own, keep=_keep_own, attend=_attend_own)[op](s)
    return dict(penalties=_penalties_plain, write=_write_plain, keep=_keep_plain, attend=_attend_plain)[op](s)


# ---- the framework's calls

def _penalties_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    return sv.penalize(s["logits"], s["history"], s["history_len"], s["tokens"], s["parent"], s["node_start"],
                       prompt_len=s["prompt_len"], repetition=s["repetition"], frequency=s["frequency"],
                       presence=s["presence"], bias=s["bias"], mask=s["mask"], mask_row=s["mask_row"], out=s["out"])


def _write_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    sv.cache_write(s["cache"], s["k"], s["v"], s["table"], s["context"], s["node_start"], max_nodes=s["max_nodes"])
    return s["cache"]


def _keep_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    context = sv.cache_keep(s["cache"], s["path"], s["accepted_len"], s["table"], s["context"])
    return s["cache"], context


def _attend_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    return sv.attend_tree(s["q"], s["cache"], s["table"], s["context"], s["node_start"], s["parent"], scale=s["scale"],
                          max_nodes=s["max_nodes"], out=s["out"])


# ---- the plain forms

def _rows_of(s):
    """Sequence of each row, and its place: 0 is the root, 1 + i node i."""
    start = s["node_start"].long()
    n = start[1:] - start[:-1] + 1
    seq = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["total"] + len(n))
    return seq, torch.arange(s["total"] + len(n), device="cuda") - start[seq] - seq


def _penalties_plain(s):
    case, v, depth = s["case"], s["case"]["v"], s["depth"]
    seq, place = _rows_of(s)
    start = s["node_start"].long()
    where = torch.arange(case["cap"], device="cuda")
    inside = where < s["history_len"].unsqueeze(1)
    prompt = where < s["prompt_len"].unsqueeze(1)
    token = s["history"].long()
    said = torch.zeros(case["b"], v + 1, dtype=torch.int32, device="cuda")
    one = torch.ones_like(token, dtype=torch.int32)
    said.scatter_add_(1, torch.where(inside & ~prompt, token, v), one)
    asked = torch.zeros(case["b"], v + 1, dtype=torch.bool, device="cuda")
    asked.scatter_(1, torch.where(inside & prompt, token, v), True)
    count = said[seq]
    cur = place - 1
    for _ in range(depth):
        node = torch.where(cur >= 0, start[seq] + cur, 0)
        at = torch.where(cur >= 0, s["tokens"].long()[node], v)
        count.scatter_add_(1, at.unsqueeze(1), torch.ones_like(at, dtype=torch.int32).unsqueeze(1))
        cur = torch.where(cur >= 0, s["parent"].long()[node], -1)
    n = count[:, :v]
    z = s["logits"].float()
    if s["repetition"] is not None:
        rep = s["repetition"][seq].unsqueeze(1)
        z = torch.where((n > 0) | asked[seq, :v], torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][seq].unsqueeze(1) * n
    z = torch.where(n > 0, z - s["presence"][seq].unsqueeze(1), z)
    if s["bias"] is not None:
        first, at, value = s["bias"]
        owner = torch.repeat_interleave(torch.arange(case["b"], device="cuda"), (first[1:] - first[:-1]).long(),
                                        output_size=len(at))
        last = torch.full((case["b"] * v,), -1, dtype=torch.int64, device="cuda")
        last.scatter_reduce_(0, owner * v + at, torch.arange(len(at), device="cuda"), "amax")  # the last one counts
        dense = torch.where(last >= 0, value[last.clamp(min=0)], 0.0).view(case["b"], v)
        z = z + dense[seq]
    if s["mask"] is not None:
        bit = torch.arange(v, device="cuda")
        word = s["mask"][s["mask_row"].long().clamp(min=0)][:, bit // 32]
        z = torch.where((((word >> (bit % 32)) & 1) == 0) & (s["mask_row"] >= 0).unsqueeze(1), -math.inf, z)
    s["out"].copy_(z)
    return s["out"]


def _need(largest):
    """The power of two that brings values of up to `largest` to 448 at most, 2^-100 at least."""
    m, e = torch.frexp(largest)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.ldexp(torch.ones_like(largest), torch.where(largest > 0, k.clamp(min=-100), -100))


def _where_at(s, seq, pos):
    """Page and place in it of a position of a sequence."""
    page = s["case"]["page"]
    return s["table"].long()[seq, pos // page], pos % page


def _byte(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _value(bytes_):
    return bytes_.contiguous().view(torch.float8_e4m3fn).float()


def _write_plain(s):
    case, block = s["case"], s["case"]["block"]
    seq, place = _rows_of(s)
    context = s["context"].long()
    pages, at = _where_at(s, seq, context[seq] + place)
    # positions of the block that the first new row falls into: the only one with older rows
    edge = (context // block * block).unsqueeze(1) + torch.arange(block, device="cuda")
    older = edge < context.unsqueeze(1)
    epage, eat = _where_at(s, torch.arange(case["b"], device="cuda").unsqueeze(1), edge)
    for x, entries, scales in ((s["k"].float(), s["cache"][0], s["cache"][2]), (s["v"].float(), s["cache"][1], s["cache"][3])):
        heads, per = x.shape[1], scales.shape[-1]
        slot = pages * per + at // block
        largest = torch.zeros(scales.shape[0] * per, heads, device="cuda")
        largest.scatter_reduce_(0, slot.unsqueeze(1).expand(-1, heads), x.abs().amax(2), "amax")
        need = _need(largest)
        flat = scales.transpose(1, 2).reshape(-1, heads)  # [pages * blocks, heads]
        new = need.clone()
        eslot = epage[:, 0] * per + eat[:, 0] // block
        had = older.any(1)
        new[eslot[had]] = torch.maximum(flat[eslot[had]], need[eslot[had]])
        old, up = flat[eslot], new[eslot]
        bytes_ = entries.view(torch.uint8)
        q = _value(bytes_[epage, :, eat]) * old[:, None, :, None] * (1.0 / up)[:, None, :, None]
        bytes_[epage, :, eat] = torch.where((older[:, :, None] & (up > old)[:, None, :])[..., None], _byte(q),
                                            bytes_[epage, :, eat])
        bytes_[pages, :, at] = _byte(x * (1.0 / new[slot]).unsqueeze(2))
        done = torch.zeros(scales.shape[0] * per, dtype=torch.bool, device="cuda")
        done[slot] = True
        flat = torch.where(done.unsqueeze(1), new, flat)
        scales.copy_(flat.view(scales.shape[0], per, heads).transpose(1, 2))
    return s["cache"]


def _keep_plain(s):
    case, block = s["case"], s["case"]["block"]
    b, depth, context = case["b"], s["depth"], s["context"].long()
    length = s["accepted_len"].long()
    some = torch.arange(b, device="cuda").unsqueeze(1)
    first = context + 1  # of the drafts
    # every position of the blocks that receive rows: those in front of the first draft stay, the others come from elsewhere
    begin = first // block * block
    pos = begin.unsqueeze(1) + torch.arange((depth // block + 2) * block, device="cuda")
    t = pos - first.unsqueeze(1)
    taken = (t >= 0) & (t < length.unsqueeze(1))
    kept = ((t < 0) & (length > 0).unsqueeze(1)) | taken
    source = torch.where(taken, first.unsqueeze(1) + s["path"].long()[some, t.clamp(0, depth - 1)], pos)
    limit = s["table"].shape[1] * case["page"] - 1
    dpage, dat = _where_at(s, some, pos.clamp(max=limit))
    spage, sat = _where_at(s, some, torch.where(kept, source, 0))
    for entries, scales in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        bytes_ = entries.view(torch.uint8)
        old = scales[:, spage, :, sat // block].movedim(2, 0)  # [layers, b, positions, heads]
        old = torch.where(kept[None, :, :, None], old, 0.0)
        most = old.unflatten(2, (-1, block)).amax(3, keepdim=True).expand(-1, -1, -1, block, -1).flatten(2, 3)
        q = _value(bytes_[:, spage, :, sat].movedim(2, 0))
        q = _byte(q * torch.where(most > 0, old / most, 1.0).unsqueeze(-1))
        at = kept.nonzero(as_tuple=True)
        bytes_[:, dpage[at], :, dat[at]] = q[:, at[0], at[1]].transpose(0, 1)
        scales[:, dpage[at], :, dat[at] // block] = most[:, at[0], at[1]].transpose(0, 1)
    return s["cache"], (context + 1 + length).to(torch.int32)


def _visible(s, rows):
    """[b, rows, rows]: whether row i's path (the root, ancestors, itself) holds row j."""
    start, b = s["node_start"].long(), s["case"]["b"]
    n = start[1:] - start[:-1]
    i = torch.arange(rows, device="cuda")
    up = torch.where((i >= 1) & (i <= n.unsqueeze(1)), (start[:-1].unsqueeze(1) + i - 1).clamp(0, max(0, s["total"] - 1)), -1)
    parent = torch.cat([s["parent"].long(), torch.full((1,), -1, device="cuda")])
    up = torch.where(up >= 0, parent[up] + 1, -1)  # the row in front of a row
    seen = torch.zeros(b, rows, rows, dtype=torch.bool, device="cuda")
    cur = i.expand(b, rows)
    for _ in range(s["depth"] + 1):
        seen |= i == cur.unsqueeze(2)
        cur = torch.where(cur >= 0, up.gather(1, cur.clamp(min=0)), -1)
    return seen


def _attend_plain(s):
    case = s["case"]
    b, heads, group, dim, block = (case[f] for f in ("b", "heads", "group", "dim", "block"))
    seq, place = _rows_of(s)
    rows = s["max_nodes"] + 1
    k, v = (_value(entries.view(torch.uint8)[s["table"].long()]).unflatten(3, (-1, block)) *
            scales[s["table"].long()][..., None, None] for entries, scales in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))
    k, v = (x.flatten(3, 4).transpose(1, 2).flatten(2, 3) for x in (k, v))  # [b, heads, positions, dim]
    q = torch.zeros(b, rows, heads, group, dim, device="cuda")
    q[seq, place] = s["q"].float().unflatten(1, (heads, group))
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [b, heads, rows * group, dim]
    scores = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (rows, group)) * s["scale"]
    pos = torch.arange(k.shape[2], device="cuda") - s["context"].long().unsqueeze(1)  # from the root on
    seen = _visible(s, rows).gather(2, pos.clamp(0, rows - 1).unsqueeze(1).expand(-1, rows, -1))
    seen = (seen & (pos < rows).unsqueeze(1)) | (pos < 0).unsqueeze(1)
    scores = torch.where(seen[:, None, :, None, :], scores, -math.inf)
    # rows that a sequence does not have see at least themselves, or nothing: they are left out at the end
    e = torch.exp(scores - scores.amax(-1, keepdim=True).clamp(min=-1e30))
    o = torch.matmul(e.flatten(2, 3), v) / e.sum(-1).clamp(min=1e-30).flatten(2, 3).unsqueeze(-1)
    o = o.unflatten(2, (rows, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s["out"].copy_(o[seq, place])
    return s["out"]


def work(case):
    b, N = case["b"], len(_parents(case["widths"])[0])
    if case["op"] == "penalties":
        nodes = N * (0.75 if case["ragged"] else 1.0)
        rows, tokens = b * (nodes + 1), case["cap"] * (0.75 if case["ragged"] else 1.0)
        es = 2 if case["dtype"] == "bf16" else 4
        if case["out"] == "same" and not case["masks"]:
            # the entries of the histories' different tokens (about half of those said twice) and of the biases
            touched = min(case["v"], tokens / 2) + case["biases"]
            return dict(bytes=b * tokens * 4 + rows * touched * 2 * es + b * case["biases"] * 8, flops=4.0 * rows * touched)
        eo = es if case["out"] == "same" else 2 if case["out"] == "bf16" else 4
        e = rows * case["v"]
        return dict(bytes=e * (es + eo) + (e / 8 if case["masks"] else 0) + b * tokens * 4, flops=2.0 * e)
    entry = case["heads"] * case["dim"]
    if case["op"] == "write":
        rows = b * (case["rows"] * 0.75 if case["rows"] else N + 1)
        return dict(bytes=2 * rows * entry * ((2 if case["dtype"] == "bf16" else 4) + 1), flops=4.0 * rows * entry)
    if case["op"] == "keep":
        depth = len(case["widths"].split(","))
        rows = b * depth / 2.0 * case["layers"]
        return dict(bytes=2 * rows * entry * 2, flops=2.0 * rows * entry)
    part = 0.75 if case["ragged"] else 1.0
    positions, rows = case["context"] * part, N * part + 1
    size = b * positions * case["heads"] * (2 * case["dim"] + 8.0 / case["block"])
    size += b * rows * entry * case["group"] * 4
    return dict(bytes=size, flops=4.0 * b * rows * entry * case["group"] * positions)


# ---- the definitions in 64 bits, sequence by sequence

def exact(case, seed):
    s = prepare(case, seed)
    return dict(penalties=_exact_penalties, write=_exact_write, keep=_exact_keep, attend=_exact_attend)[case["op"]](s)


def _paths(s):
    """For each sequence the first row, and for each of its rows the nodes from the root's child down to it."""
    start, parent = s["node_start"].tolist(), s["parent"].tolist()
    for q, (lo, hi) in enumerate(zip(start[:-1], start[1:])):
        paths = [[]]
        for i in range(hi - lo):
            paths.append(paths[1 + parent[lo + i]] + [i])
        yield q, lo, paths


def _exact_penalties(s):
    v = s["case"]["v"]
    out = s["logits"].double()
    lens, prompts = s["history_len"].tolist(), s["prompt_len"].tolist()
    for q, lo, paths in _paths(s):
        words = s["history"][q].long()
        base = torch.bincount(words[prompts[q]:lens[q]], minlength=v)
        prompt = torch.bincount(words[:prompts[q]], minlength=v) > 0
        bias = torch.zeros(v, dtype=torch.float64, device="cuda")
        if s["bias"] is not None:
            first, at, value = (t.tolist() for t in s["bias"])
            last = {at[j]: value[j] for j in range(first[q], first[q + 1])}
            bias[torch.tensor(list(last), device="cuda")] = torch.tensor(list(last.values()), dtype=torch.float64, device="cuda")
        for i, path in enumerate(paths):
            z = out[lo + q + i]
            n = base
            if path:
                n = n + torch.bincount(s["tokens"].long()[lo + torch.tensor(path, device="cuda")], minlength=v)
            if s["repetition"] is not None:
                rep = float(s["repetition"][q])
                z = z * torch.where((n > 0) | prompt, torch.where(z > 0, 1.0 / rep, rep), 1.0)
            z = z + bias - float(s["frequency"][q]) * n - float(s["presence"][q]) * (n > 0)
            if s["mask"] is not None and int(s["mask_row"][lo + q + i]) >= 0:
                word = s["mask"][int(s["mask_row"][lo + q + i])].long()
                bits = (word.unsqueeze(1) >> torch.arange(32, device="cuda")).bitwise_and(1).flatten()[:v]
                z = torch.where(bits == 1, z, -math.inf)
            out[lo + q + i] = z
    return out


def _exact_write(s):
    case, page, block = s["case"], s["case"]["page"], s["case"]["block"]
    start, context, table = s["node_start"].tolist(), s["context"].tolist(), s["table"].tolist()
    got = []
    for x, entries, scales in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        values, sizes = entries.double(), scales.double()
        for q in range(case["b"]):
            lo, c = start[q] + q, context[q]
            end = c + start[q + 1] - start[q] + 1
            for p in range(c // block * block, end, block):
                pg, at = table[q][p // page], p % page
                new = x[lo + max(p, c) - c:lo + min(p + block, end) - c].double()  # [rows, heads, dim]
                most = new.abs().amax((0, 2))
                need = torch.exp2((torch.round(torch.log2(most)) - 10.0).clamp(min=-100.0))
                for _ in range(3):  # the logarithm may be off where the answer turns
                    need = torch.where(need * 448.0 < most, need * 2.0, need)
                old = sizes[pg, :, at // block]
                size = torch.maximum(need, old) if p < c else need
                if p < c:
                    values[pg, :, at:at + c - p] *= (old / size)[:, None, None]
                f = at + max(p, c) - p
                values[pg, :, f:f + len(new)] = new.transpose(0, 1) / size[:, None, None]
                sizes[pg, :, at // block] = size
        got.append((values, sizes))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def _exact_keep(s):
    case, page, block = s["case"], s["case"]["page"], s["case"]["block"]
    context, table = s["context"].tolist(), s["table"].tolist()
    path, length = s["path"].tolist(), s["accepted_len"].tolist()
    got = []
    for entries, scales in ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])):
        values, sizes = entries.double(), scales.double()
        for q in range(case["b"]):
            first = context[q] + 1
            end = first + length[q]
            place = lambda p: (table[q][p // page], p % page)  # noqa: B023, E731
            for p in range(first // block * block, end if length[q] else 0, block):
                rows = [(d, d if d < first else first + path[q][d - first]) for d in range(p, min(p + block, end))]
                from_ = [place(r) for _, r in rows]
                old = [sizes[:, pg, :, at // block].clone() for pg, at in from_]
                held = [values[:, pg, :, at].clone() for pg, at in from_]
                size = torch.stack(old).amax(0)
                for (d, _), o, h in zip(rows, old, held):
                    pg, at = place(d)
                    values[:, pg, :, at] = h * (o / size).unsqueeze(-1)
                pg, at = place(p)
                sizes[:, pg, :, at // block] = size
        got.append((values, sizes))
    return (got[0][0], got[1][0], got[0][1], got[1][1]), None


def _exact_attend(s):
    case = s["case"]
    heads, group, block = case["heads"], case["group"], case["block"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    context = s["context"].tolist()
    for q, lo, paths in _paths(s):
        c = context[q]
        pages = s["table"][q].long()
        k, v = ((_value(entries.view(torch.uint8)[pages]).double().unflatten(2, (-1, block)) *
                 scales[pages].double()[..., None, None]).flatten(2, 3).transpose(0, 1).flatten(1, 2) for entries, scales in
                ((s["cache"][0], s["cache"][2]), (s["cache"][1], s["cache"][3])))  # [heads, positions, dim]
        seen = torch.zeros(len(paths), c + len(paths), dtype=torch.bool, device="cuda")
        seen[:, :c + 1] = True
        for i, path in enumerate(paths):
            if path:
                seen[i, c + 1 + torch.tensor(path, device="cuda")] = True
        x = s["q"][lo + q:lo + q + len(paths)].double().unflatten(1, (heads, group))
        scores = torch.einsum("rhgd,hpd->hrgp", x, k[:, :c + len(paths)]) * s["scale"]
        scores = scores.masked_fill(~seen[None, :, None, :], -math.inf)
        o = torch.einsum("hrgp,hpd->rhgd", torch.softmax(scores, -1), v[:, :c + len(paths)])
        out[lo + q:lo + q + len(paths)] = o.flatten(1, 2)
    return out
