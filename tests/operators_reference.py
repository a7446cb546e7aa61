"""Plain 64-bit implementations of the operators around a verifying call, and
the inputs their tests share.  Written from the header's text: the residual
distribution is carried along as such, node by node."""
from __future__ import annotations

import math

import numpy as np
import torch

UNREACHED, ACCEPT, REJECT, INVALID = 0, 1, 2, 4


def pick(weights, u):
    """Smallest index whose inclusive prefix sum exceeds u * total; the last weight where none does."""
    sums = np.cumsum(weights)
    past = np.nonzero(sums > u * sums[-1])[0]
    return int(past[0]) if len(past) else int(np.nonzero(weights > 0)[0][-1])


def tree(p, q, tokens, parent, draft_row, node_start, u_accept, u_pick, max_nodes, max_depth, replacement=True):
    """numpy arrays in, the dict of verify_tree out (accept_prob in 64 bits), and counters [8]."""
    B, total, V = len(u_pick), len(tokens), p.shape[1]
    out = dict(accepted_len=np.full(B, -1, np.int32), tokens=np.full((B, max_depth + 1), -1, np.int32),
               path=np.full((B, max_depth), -1, np.int32), accept_prob=np.zeros(total), flags=np.zeros(total, np.int8))
    cnt = np.zeros(8, np.int64)
    for b in range(B):
        lo, hi = int(node_start[b]), int(node_start[b + 1])
        n = hi - lo
        if lo < 0 or hi < lo or hi > total or n > max_nodes:
            cnt[6] += 1
            if 0 <= lo <= hi <= total:
                out["flags"][lo:hi] = INVALID
            continue
        res = _tree_one(p[lo + b:hi + b + 1], q, tokens[lo:hi], parent[lo:hi], draft_row[lo + b:hi + b + 1],
                        u_accept[lo:hi].astype(np.float64), float(u_pick[b]), max_depth, replacement, V)
        if res is None:
            cnt[6] += 1
            out["flags"][lo:hi] = INVALID
            continue
        path, tok, alpha, flags, bonus, degenerate = res
        out["accepted_len"][b] = len(path)
        out["path"][b, :len(path)] = path
        out["tokens"][b, :len(path)] = tokens[lo:hi][path]
        out["tokens"][b, len(path)] = tok
        out["accept_prob"][lo:hi], out["flags"][lo:hi] = alpha, flags
        cnt[0] += int((flags != 0).sum())
        cnt[1] += len(path)
        cnt[3] += int((flags == REJECT).sum())
        cnt[4] += bonus
        cnt[7] += degenerate
    return out, cnt


def _tree_one(p, q, tokens, parent, draft_row, u, u_pick, max_depth, replacement, V):
    n = len(tokens)
    depth = []
    rows_q = 0 if q is None else q.shape[0]
    if np.any(draft_row < -1) or np.any(draft_row >= rows_q):
        return None
    for i in range(n):
        if not 0 <= tokens[i] < V or not -1 <= parent[i] < i:
            return None
        depth.append(1 if parent[i] < 0 else depth[parent[i]] + 1)
        if depth[i] > max_depth:
            return None
    alpha, flags, path = np.zeros(n), np.zeros(n, np.int8), []
    cur = -1
    while True:
        row = p[cur + 1].astype(np.float64)
        certain = draft_row[cur + 1] < 0
        prop = None if certain else q[draft_row[cur + 1]].astype(np.float64)
        rest, Z, offered = row.copy(), 1.0, 0.0  # rest / Z is the distribution
        children = [i for i in range(n) if parent[i] == cur]
        chosen = None
        for i in children:
            x = tokens[i]
            if not (np.isfinite(row[x]) and row[x] >= 0):
                return None
            if certain:
                mu_x = 1.0
            else:
                if not (np.isfinite(prop[x]) and prop[x] >= 0):
                    return None
                w = 1.0 if replacement else max(1.0 - offered, prop[x])
                mu_x = prop[x] / w if w > 0 else 0.0
            ok = rest[x] > 0 and u[i] * mu_x * Z <= rest[x]
            if mu_x * Z > 0:
                alpha[i] = min(1.0, rest[x] / (mu_x * Z))
            else:
                alpha[i] = float(rest[x] > 0)
            flags[i] = ACCEPT if ok else REJECT
            if ok:
                chosen = i
                break
            if certain:
                Z -= rest[x]
                rest[x] = 0.0
            else:
                if not (np.all(np.isfinite(row)) and np.all(np.isfinite(prop))):
                    return None
                if w > 0:
                    rest = np.maximum(rest - Z * (prop / w), 0.0)
                Z = math.fsum(rest)
                offered += prop[x]
        if chosen is None:
            break
        path.append(chosen)
        cur = chosen
    degenerate = 0
    if np.isfinite(rest).all() and rest.sum() == 0.0:
        degenerate, rest = 1, row
    if not np.isfinite(rest).all() or not rest.sum() > 0:
        return None
    return np.array(path, int), pick(rest, u_pick), alpha, flags, int(not children), degenerate


def random_tree_batch(seed, B, V, max_nodes, max_depth, replacement, kind="sampled", sharp=2.0, noise=0.7, shape="any",
                      pad=0):
    """A seeded batch of random trees: node i hangs on a random earlier node (shape "any"), on node i - 1
    ("chain") or on the root ("star"); rows are softmaxes of normal logits, tokens drawn from the rows' proposals.
    kind: sampled, certain, or mixed (row by row).  pad: extra entries behind each row."""
    rng = np.random.default_rng(seed)
    n = rng.integers(0, max_nodes + 1, B)
    start = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    total = int(start[-1])
    R = total + B
    logits = rng.standard_normal((R, V)) * sharp
    p = _softmax(logits).astype(np.float32)
    q = _softmax(logits + noise * rng.standard_normal((R, V))).astype(np.float32)
    parent, tokens = np.zeros(total, np.int32), np.zeros(total, np.int32)
    draft_row = np.arange(R, dtype=np.int32)
    certain = {"sampled": 0.0, "certain": 1.0, "mixed": 0.4}[kind]
    draft_row[rng.random(R) < certain] = -1
    for b in range(B):
        depth = []
        for i in range(n[b]):
            if shape == "chain":
                a = i - 1
            elif shape == "star":
                a = -1
            else:
                a = int(rng.integers(-1, i))
            while a >= 0 and depth[a] >= max_depth:
                a = int(parent[start[b] + a])
            parent[start[b] + i] = a
            depth.append(1 if a < 0 else depth[a] + 1)
            row = start[b] + b + 1 + a
            dist = q[row].astype(np.float64)
            if not replacement:
                for j in range(i):
                    if parent[start[b] + j] == a and draft_row[row] >= 0:
                        dist[tokens[start[b] + j]] = 0.0
            if dist.sum() <= 0:
                dist = np.ones(V)
            tokens[start[b] + i] = rng.choice(V, p=dist / dist.sum()) if V <= 4096 else pick(dist, rng.random())
    u_accept = rng.random(total).astype(np.float32)
    u_accept = np.minimum(u_accept, np.float32(1 - 2.0 ** -24))
    u_pick = np.minimum(rng.random(B).astype(np.float32), np.float32(1 - 2.0 ** -24))
    perm = rng.permutation(R)  # the proposals' rows in another order than the targets'
    q_shuffled = np.empty_like(q)
    q_shuffled[perm] = q
    draft_row = np.where(draft_row >= 0, perm[draft_row], -1).astype(np.int32)
    return dict(p=p, q=q_shuffled, tokens=tokens, parent=parent, draft_row=draft_row, node_start=start,
                u_accept=u_accept, u_pick=u_pick)


def _softmax(x):
    e = np.exp(x - x.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def on_gpu(batch, pad=0, offset=0):
    """The batch's arrays as device tensors; probability rows ``pad`` entries further apart than their length, the
    first one ``offset`` entries into its storage."""
    t = {}
    for name, a in batch.items():
        if name in ("p", "q") and (pad or offset):
            R, V = a.shape
            store = torch.full((offset + R * (V + pad),), float("nan"), device="cuda")
            view = store[offset:].view(R, V + pad)[:, :V]
            view.copy_(torch.as_tensor(a))
            t[name] = view
        else:
            t[name] = torch.as_tensor(a).cuda()
    return t


ACT = {
    "none": lambda z, cap: z,
    "relu": lambda z, cap: torch.clamp(z, min=0.0),
    "silu": lambda z, cap: z * torch.sigmoid(z),
    "gelu": lambda z, cap: 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0)),
    "gelu_tanh": lambda z, cap: 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))),
    "softcap": lambda z, cap: cap * torch.tanh(z / cap),
}


def linear(x, w, bias, residual, act, cap):
    """(y, bound): the result in 64 bits and how far an fp32 evaluation may be from it before its last rounding.

    Every addition of a product is off by at most a step of the running sum, 2^-23 of sum |x w| (a half when it
    rounds to nearest, one when it truncates), so the sum by K * 2^-23 * sum |x w|.  The activations' slopes are
    below 1.2; they and the remaining additions are a few operations and one library function of at most 4 steps,
    taken together as 16 half steps of |z| + |bias| + |residual| + 1."""
    x, w = x.double(), w.double()
    K = x.shape[-1]
    z = torch.matmul(x, w.transpose(-1, -2))
    mag = torch.matmul(x.abs(), w.abs().transpose(-1, -2))
    size = z.abs() + 1.0
    if bias is not None:
        b = bias.double().unsqueeze(-2)
        z, size = z + b, size + b.abs()
    y = ACT[act](z, cap)
    if residual is not None:
        y, size = y + residual.double(), size + residual.double().abs()
    return y, 1.2 * K * 2.0 ** -23 * mag + 16 * 2.0 ** -24 * size


def assert_linear(got, x, w, bias, residual, act, cap, what=""):
    y, bound = linear(x, w, bias, residual, act, cap)
    half = torch.finfo(got.dtype).eps / 2
    # y is rounded once: by half a step of a value that may itself be `bound` off
    bound = bound + half * (y.abs() + bound)
    off = (got.double() - y).abs()
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert bool((off <= bound).all()), f"{what}: {worst:.3g} of the bound, off by up to {float(off.max()):.3g}"
    return worst
