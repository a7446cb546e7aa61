"""Cases of the operators around a verification call: the matrix product of the
draft blocks and output heads, the probabilities of logits rows, and the
verification of drafted trees against probabilities from given uniforms.

``run`` computes them with elementary torch operations where ``own`` is false
and through the package's entry points where it is true.
"""
import math

import torch

own = False

MAX_WORK = 6.0e11  # floating point operations of the largest matrix product drawn


def listed():
    return [
        # draft blocks of one sequence, four heads: the smallest call
        dict(name="blocks_m1", op="linear", groups=4, m=1, n=2048, k=2048, out="bf16", act="silu", bias=True,
             residual=True, shared=True, pad=0),
        # draft blocks of a batch of 64 with five heads
        dict(name="blocks_m64", op="linear", groups=5, m=64, n=4096, k=4096, out="bf16", act="silu", bias=True,
             residual=True, shared=True, pad=0),
        # the target's output head for one sequence with five drafts
        dict(name="head_m6_v151936", op="linear", groups=1, m=6, n=151936, k=2048, out="f32", act="none", bias=False,
             residual=False, shared=False, pad=0),
        # the target's output head for 64 sequences with five drafts
        dict(name="head_m384_v128256", op="linear", groups=1, m=384, n=128256, k=4096, out="bf16", act="softcap",
             bias=False, residual=False, shared=False, pad=0),
        # 256 sequences with eight drafts: bound by the tensor cores
        dict(name="head_m2304_v32000", op="linear", groups=1, m=2304, n=32000, k=4096, out="bf16", act="none",
             bias=True, residual=False, shared=False, pad=0),
        # nothing divides anything: rows that start at odd places
        dict(name="odd_m77_v32001", op="linear", groups=2, m=77, n=32001, k=1001, out="f32", act="gelu", bias=True,
             residual=True, shared=False, pad=3),
        # probabilities of a small batch's target rows
        dict(name="probs_r80_v32000", op="softmax", rows=80, v=32000, dtype="bf16", per_row=False),
        # and of the 128K-vocabulary batch, a temperature for each row
        dict(name="probs_r384_v128256", op="softmax", rows=384, v=128256, dtype="bf16", per_row=True),
        # few long rows of an odd length
        dict(name="probs_r7_v262143", op="softmax", rows=7, v=262143, dtype="f32", per_row=True),
        # one sequence's chain of four drafts
        dict(name="chain_b1_v32000", op="tree", b=1, widths="1,1,1,1", v=32000, ragged=False, proposal="sampled",
             replacement=True),
        # chains of up to five drafts, some of them without a draft distribution
        dict(name="chain_b64_v128256", op="tree", b=64, widths="1,1,1,1,1", v=128256, ragged=True, proposal="mixed",
             replacement=True),
        # trees of up to 21 drafts drawn without replacement
        dict(name="tree_b32_v151936", op="tree", b=32, widths="3,2,2", v=151936, ragged=True, proposal="sampled",
             replacement=False),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "softmax", "tree"])
    if op == "linear":
        groups = rng.choice([1, 1, 2, 4, 5])
        m, k = _spread(rng, 1, 2304), _spread(rng, 64, 8192)
        n = _spread(rng, 256, 262144 if groups == 1 else 32768)
        if rng.random() < 0.7:  # most model dimensions are multiples of 64
            k, n = max(64, k // 64 * 64), max(64, n // 64 * 64)
        n = max(1, min(n, int(MAX_WORK / (2.0 * groups * m * k)), int(5.2e8 / (groups * k)), int(7e7 / (groups * m))))
        return dict(op="linear", groups=groups, m=m, n=n, k=k, out=rng.choice(["bf16", "f32"]),
                    act=rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh", "softcap"]),
                    bias=rng.random() < 0.5, residual=rng.random() < 0.5, shared=rng.random() < 0.5,
                    pad=rng.choice([0, 0, 8, 3]))
    if op == "softmax":
        v = _spread(rng, 1000, 262144)
        return dict(op="softmax", rows=max(1, min(_spread(rng, 1, 4096), int(4.9e7 / v))), v=v,
                    dtype=rng.choice(["bf16", "f32"]), per_row=rng.random() < 0.5)
    v = _spread(rng, 1000, 262144)
    widths = rng.choice(["1", "1,1,1", "1,1,1,1,1,1,1,1", "4", "2,2,2", "4,2,1,1", "8,1"])
    nodes = sum(_levels(widths))
    return dict(op="tree", b=max(1, min(_spread(rng, 1, 256), int(1.07e8 / (v * (nodes + 1))))), widths=widths, v=v,
                ragged=rng.random() < 0.5, proposal=rng.choice(["sampled", "mixed", "given"]),
                replacement=rng.random() < 0.5)


def _levels(widths):
    """Nodes at each depth of the full tree."""
    sizes, n = [], 1
    for w in widths.split(","):
        n *= int(w)
        sizes.append(n)
    return sizes


def _parents(widths):
    """Parent of each node of the full tree, level by level (-1: the root), and its place among its siblings."""
    parent, place, last = [], [], [-1]
    for w in widths.split(","):
        level = []
        for node in last:
            for j in range(int(w)):
                level.append(len(parent))
                parent.append(node)
                place.append(j)
        last = level
    return parent, place


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "linear":
        return _prepare_linear(case, g)
    if case["op"] == "softmax":
        return _prepare_softmax(case, g)
    return _prepare_tree(case, g)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _prepare_linear(case, g):
    G, m, n, k, pad = (case[f] for f in ("groups", "m", "n", "k", "pad"))
    x = torch.randn(1 if case["shared"] else G, m, k + pad, generator=g, device="cuda")
    x = x.to(torch.bfloat16)[:, :, :k]
    w = torch.empty(G, n, k + pad, dtype=torch.bfloat16, device="cuda")
    w.normal_(0.0, 1.0 / math.sqrt(k), generator=g)
    s = dict(case=case, x=x[0] if case["shared"] else x, w=w[:, :, :k], bias=None, residual=None)
    if case["bias"]:
        s["bias"] = (torch.randn(G, n, generator=g, device="cuda") * 0.5).to(torch.bfloat16)
    if case["residual"]:
        # hidden states of [batch, heads, n], seen head by head
        r = torch.randn(m, G, n, generator=g, device="cuda").to(torch.bfloat16)
        s["residual"] = r.transpose(0, 1)
    # results as [batch, heads, n], the verifier's layout of draft rows
    s["out"] = torch.empty(m, G, n, dtype=_dtype(case["out"]), device="cuda").transpose(0, 1)
    return s


def _prepare_softmax(case, g):
    rows, v = case["rows"], case["v"]
    x = torch.randn(rows, v, generator=g, device="cuda") * 3.0
    t = 0.6
    if case["per_row"]:
        t = torch.rand(rows, generator=g, device="cuda") + 0.5
    return dict(case=case, logits=x.to(_dtype(case["dtype"])), t=t,
                out=torch.empty(rows, v, dtype=torch.float32, device="cuda"))


def _prepare_tree(case, g):
    dev = "cuda"
    B, v = case["b"], case["v"]
    parent1, place1 = (torch.tensor(a, device=dev) for a in _parents(case["widths"]))
    N, depth = len(parent1), len(case["widths"].split(","))
    width = max(int(w) for w in case["widths"].split(","))
    n = torch.full((B,), N, device=dev)
    if case["ragged"]:
        # the same lengths for every seed, in another order
        n = (N + 1) // 2 + torch.randperm(B, generator=g, device=dev) % (N - (N + 1) // 2 + 1)
    start = torch.zeros(B + 1, dtype=torch.int64, device=dev)
    start[1:] = n.cumsum(0)
    total = int(start[-1])
    seq = torch.repeat_interleave(torch.arange(B, device=dev), n)
    idx = torch.arange(total, device=dev) - start[seq]
    parent, place = parent1[idx], place1[idx]
    row_of_parent = start[seq] + seq + 1 + parent
    R = total + B
    logits = torch.randn(R, v, generator=g, device=dev) * 3.0
    peak = torch.randint(0, v, (R, 4), generator=g, device=dev)
    logits.scatter_add_(1, peak, 8.0 * torch.rand(R, 4, generator=g, device=dev))
    draft_row = torch.full((R,), -1, dtype=torch.int64, device=dev)
    inner = torch.unique(row_of_parent)
    draft_row[inner] = torch.arange(len(inner), device=dev)
    q = torch.softmax(logits[inner] + 0.8 * torch.randn(len(inner), v, generator=g, device=dev), 1)
    p = torch.softmax(logits, 1)
    del logits
    if case["replacement"]:
        drawn = torch.multinomial(q, width, replacement=True, generator=g)
    else:
        e = torch.empty_like(q).exponential_(generator=g)
        drawn = torch.topk(q / e, min(width, v), dim=1).indices
    tokens = drawn[draft_row[row_of_parent], place]
    # proposals without a distribution: a given share of the sequences
    share = dict(sampled=0.0, mixed=0.3, given=1.0)[case["proposal"]]
    bare = torch.rand(B, generator=g, device=dev) < share
    row_seq = torch.repeat_interleave(torch.arange(B, device=dev), n + 1)
    draft_row = torch.where(bare[row_seq], -1, draft_row)
    i32 = lambda a: a.to(torch.int32).contiguous()  # noqa: E731
    return dict(case=case, p=p, q=q, tokens=i32(tokens), parent=i32(parent), draft_row=i32(draft_row),
                node_start=i32(start), u=torch.rand(total, generator=g, device=dev),
                u_pick=torch.rand(B, generator=g, device=dev), max_nodes=N, max_depth=depth)


def run(s):
    op = s["case"]["op"]
    if op == "linear":
        return _linear_own(s) if own else _linear_plain(s)
    if op == "softmax":
        return _softmax_own(s) if own else _softmax_plain(s)
    return _tree_own(s) if own else _tree_plain(s)


CAP = 30.0  # of the soft cap


def _linear_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    return sv.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], activation=s["case"]["act"], cap=CAP,
                     out=s["out"])


def _activate(y, act):
    if act == "relu":
        return torch.where(y > 0, y, 0.0)
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if act == "softcap":
        return CAP * torch.tanh(y / CAP)
    return y


def _linear_plain(s):
    y = torch.matmul(s["x"].float(), s["w"].float().mT)
    if s["bias"] is not None:
        y = y + s["bias"].float().unsqueeze(1)
    y = _activate(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    s["out"].copy_(y)
    return s["out"]


def _softmax_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    return sv.softmax(s["logits"], s["t"], out=s["out"])


def _softmax_plain(s):
    t = s["t"] if isinstance(s["t"], float) else s["t"].unsqueeze(1)
    x = s["logits"].float()
    e = torch.exp((x - x.amax(1, keepdim=True)) / t)
    s["out"].copy_(e / e.sum(1, keepdim=True))
    return s["out"]


def _tree_own(s):
    import speculative_decoding_verification_online_gb300 as sv
    return sv.verify_tree(s["p"], s["q"], s["tokens"], s["parent"], s["draft_row"], s["node_start"], s["u"],
                          s["u_pick"], max_nodes=s["max_nodes"], max_depth=s["max_depth"],
                          replacement=s["case"]["replacement"])


def _tree_plain(s):
    """Every sequence's walk at once, node by node in index order; sums in 64 bits, for a pick over the vocabulary
    hangs on the last digits of its prefix sums."""
    p, q, v, dev = s["p"], s["q"], s["case"]["v"], s["p"].device
    B, N, replacement = s["case"]["b"], s["max_nodes"], s["case"]["replacement"]
    start = s["node_start"].long()
    n, start = start[1:] - start[:-1], start[:-1]
    at = start.unsqueeze(1) + torch.arange(N, device=dev)
    there = torch.arange(N, device=dev) < n.unsqueeze(1)
    at = torch.where(there, at, 0)
    tokens, parent = s["tokens"].long()[at], torch.where(there, s["parent"].long()[at], -2)
    u = s["u"].double()[at]
    root = start + torch.arange(B, device=dev)
    f64 = dict(dtype=torch.float64, device=dev)
    cur = torch.full((B,), -1, dtype=torch.int64, device=dev)
    c, Z, mass = torch.zeros(B, **f64), torch.ones(B, **f64), torch.zeros(B, **f64)
    flags = torch.zeros(B, N, dtype=torch.int8, device=dev)
    alpha = torch.zeros(B, N, **f64)
    length = torch.zeros(B, dtype=torch.int64, device=dev)
    path = torch.full((B, s["max_depth"]), -1, dtype=torch.int32, device=dev)
    out_tokens = torch.full((B, s["max_depth"] + 1), -1, dtype=torch.int32, device=dev)
    some = torch.arange(B, device=dev)

    def residual():
        row = root + 1 + cur
        return torch.clamp(p[row].double() - c.unsqueeze(1) * q[s["draft_row"].long()[row].clamp(min=0)].double(),
                           min=0.0)

    for i in range(N):
        has = parent[:, i] == cur
        row, x = root + 1 + cur, tokens[:, i]
        d = s["draft_row"].long()[row]
        bare = d < 0
        again = ((flags == 2) & (parent == cur.unsqueeze(1)) & (tokens == x.unsqueeze(1))).any(1)
        px = torch.where(bare & again, 0.0, p[row, x].double())
        qx = torch.where(bare, 1.0, q[d.clamp(min=0), x].double())
        r = torch.clamp(px - torch.where(bare, 0.0, c) * qx, min=0.0)
        w = torch.ones_like(qx) if replacement else torch.where(bare, 1.0, torch.maximum(1.0 - mass, qx))
        yes = has & (r > 0) & (u[:, i] * qx * Z <= r * w)
        no = has & ~yes
        most = qx * Z
        ratio = torch.where(most > 0, torch.clamp(r * w / most, max=1.0), torch.where(r > 0, 1.0, 0.0))
        alpha[:, i] = torch.where(has, ratio, 0.0)
        flags[:, i] = torch.where(yes, 1, torch.where(no, 2, 0)).to(torch.int8)
        c = torch.where(no & ~bare, torch.clamp(c + torch.where(w > 0, Z / w, 0.0), max=1e30), c)
        mass = torch.where(no, mass + qx, mass)
        Z = torch.where(no, torch.where(bare, Z - r, residual().sum(1)), Z)
        path[some, length.clamp(max=s["max_depth"] - 1)] = torch.where(
            yes, i, path[some, length.clamp(max=s["max_depth"] - 1)].long()).to(torch.int32)
        out_tokens[some, length] = torch.where(yes, x, out_tokens[some, length].long()).to(torch.int32)
        length = torch.where(yes, length + 1, length)
        cur, c, mass = torch.where(yes, i, cur), torch.where(yes, 0.0, c), torch.where(yes, 0.0, mass)
        Z = torch.where(yes, 1.0, Z)
    # a row without a draft distribution is left with the tokens not refused
    refused = (flags == 2) & (parent == cur.unsqueeze(1))
    gone = torch.zeros(B, v + 1, dtype=torch.bool, device=dev).scatter_(1, torch.where(refused, tokens, v), True)
    bare = s["draft_row"].long()[root + 1 + cur] < 0
    weights = torch.where(bare.unsqueeze(1) & gone[:, :v], 0.0, residual())
    weights = torch.where(weights.sum(1, keepdim=True) > 0, weights, p[root + 1 + cur].double())
    sums = weights.cumsum(1)
    pick = (sums <= s["u_pick"].double().unsqueeze(1) * sums[:, -1:]).sum(1)
    last = v - 1 - (weights.flip(1) > 0).to(torch.int8).argmax(1)
    out_tokens[some, length] = torch.minimum(pick, last).to(torch.int32)
    return dict(accepted_len=length.to(torch.int32), tokens=out_tokens, path=path, accept_prob=alpha[there].float(),
                flags=flags[there])


def work(case):
    if case["op"] == "linear":
        G, m, n, k = (case[f] for f in ("groups", "m", "n", "k"))
        size = 2 if case["out"] == "bf16" else 4
        b = G * n * k * 2 + (1 if case["shared"] else G) * m * k * 2 + G * m * n * size
        b += G * n * 2 * case["bias"] + G * m * n * 2 * case["residual"]
        return dict(bytes=b, flops=2.0 * G * m * n * k)
    if case["op"] == "softmax":
        e = case["rows"] * case["v"]
        return dict(bytes=e * ((2 if case["dtype"] == "bf16" else 4) + 4), flops=4.0 * e)
    # the rows that the last token is picked from: every other row is read at single tokens, or only where a
    # candidate before an accepted sibling was refused
    e = case["b"] * case["v"]
    rows = dict(sampled=2.0, mixed=1.7, given=1.0)[case["proposal"]]
    return dict(bytes=e * 4 * rows, flops=3.0 * e)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(s)
    if case["op"] == "softmax":
        t = s["t"] if isinstance(s["t"], float) else s["t"].double().unsqueeze(1)
        return torch.softmax(s["logits"].double() / t, 1)
    return dict(accepted_len=None, tokens=None, path=None, accept_prob=_exact_alpha(s), flags=None)


def _exact_linear(s):
    F = torch.nn.functional
    act = dict(none=lambda y: y, relu=F.relu, silu=F.silu, gelu=F.gelu,
               gelu_tanh=lambda y: F.gelu(y, approximate="tanh"), softcap=lambda y: CAP * torch.tanh(y / CAP))
    out = torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    for h in range(s["w"].shape[0]):
        x = s["x"] if s["x"].dim() == 2 else s["x"][h]
        y = x.double() @ s["w"][h].double().T
        if s["bias"] is not None:
            y = y + s["bias"][h].double()
        y = act[s["case"]["act"]](y)
        if s["residual"] is not None:
            y = y + s["residual"][h].double()
        out[h] = y
    return out


def _exact_alpha(s):
    """Sequence by sequence, with the residual distribution itself carried from sibling to sibling."""
    start, tokens, parent = s["node_start"].tolist(), s["tokens"].tolist(), s["parent"].tolist()
    draft_row, u = s["draft_row"].tolist(), s["u"].double().tolist()
    alpha = [0.0] * len(tokens)
    for b in range(s["case"]["b"]):
        lo, hi, cur = start[b], start[b + 1], -1
        i, rest, prop = lo, None, None
        while i < hi:
            if parent[i] != cur:
                i += 1
                continue
            if rest is None:
                row = lo + b + 1 + cur
                rest, bare = s["p"][row].double(), draft_row[row] < 0
                prop = None if bare else s["q"][draft_row[row]].double()
            x = tokens[i]
            if prop is None:
                ratio = min(1.0, float(rest[x]))
            else:
                qx = float(prop[x])
                ratio = min(1.0, float(rest[x]) / qx) if qx > 0 else float(rest[x] > 0)
            alpha[i] = ratio
            if ratio > 0 and u[i] <= ratio:
                cur, rest = i - lo, None
            elif prop is None:
                left = 1.0 - float(rest[x])
                rest = rest.clone()
                rest[x] = 0.0
                rest = rest / left
            else:
                rest = torch.clamp(rest - prop, min=0.0)
                total = float(rest.sum())
                rest = rest / total if total > 0 else rest
                if not s["case"]["replacement"]:
                    prop = prop.clone()
                    prop[x] = 0.0
                    # what is left of the proposal is taken as 1 minus what was drawn, as a sampler keeps it
                    prop = prop / max(1.0 - qx, 1e-300)
            i += 1
    return torch.tensor(alpha, dtype=torch.float64, device="cuda")
