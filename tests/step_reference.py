"""64-bit implementations of the operators around a tree's target pass, on the host, position by position: penalties, the
8-bit cache and the attention over it.  Inputs are tensors of any device."""
from __future__ import annotations

import numpy as np
import torch

# the values of the 256 e4m3 ("fn") entries
_byte = np.arange(256)
_exp, _man = (_byte >> 3) & 15, _byte & 7
E4M3 = np.where(_exp == 0, _man * 2.0 ** -9, (8 + _man) * 2.0 ** (_exp - 10.0)) * np.where(_byte & 128, -1.0, 1.0)
E4M3[[0x7f, 0xff]] = np.nan
FINITE = np.sort(np.unique(E4M3[~np.isnan(E4M3)]))


def nearest_off(x):
    """How far each value is from the e4m3 value that is nearest to it (448 beyond)."""
    x = np.clip(x, -448.0, 448.0)
    at = np.clip(np.searchsorted(FINITE, x), 1, len(FINITE) - 1)
    return np.minimum(np.abs(x - FINITE[at - 1]), np.abs(x - FINITE[at]))


def assert_rounded(entries, want, what, slack=2.0 ** -22):
    """Entries (as values) are nearest to the wanted ones, which the call may have had off by `slack` before it rounded."""
    assert np.array_equal(np.isnan(entries), np.isnan(want)), what
    fine = ~np.isnan(want)
    e, w = entries[fine], want[fine]
    off = np.abs(e - np.clip(w, -448.0, 448.0))
    assert np.all(off <= nearest_off(w) + 2 * slack * np.abs(w)), (what, float(np.max(off - nearest_off(w))))


def ints(t):
    return t.cpu().numpy().astype(np.int64)


def doubles(t):
    return t.detach().double().cpu().numpy()


def values(t):
    """float8_e4m3fn entries as values."""
    return E4M3[t.cpu().contiguous().view(torch.uint8).numpy()]


def path_of(parent, i):
    """Nodes of row i (0: the root), itself first."""
    nodes, cur = [], i - 1
    while cur >= 0:
        nodes.append(cur)
        cur = parent[cur]
    return nodes


def penalties(logits, history, history_len, tokens, parent, node_start, prompt_len=None, repetition=None, frequency=None,
              presence=None, bias=None, mask=None, mask_row=None):
    """The rows as they should be, and the sum of the magnitudes that went into each entry."""
    out, V = doubles(logits).copy(), logits.shape[1]
    size = np.abs(np.where(np.isfinite(out), out, 0.0))
    hist, start, tok = ints(history), ints(node_start), ints(tokens)
    par = None if parent is None else ints(parent)
    words = None if mask is None else mask.cpu().numpy().view(np.uint32)
    for b in range(len(start) - 1):
        n_hist = int(history_len[b])
        if n_hist < 0:
            continue
        asked = 0 if prompt_len is None else min(max(int(prompt_len[b]), 0), n_hist)
        inside = hist[b, :n_hist]
        prompt = {int(t) for t in inside[:asked]}
        base = {}
        for t in inside[asked:]:
            base[int(t)] = base.get(int(t), 0) + 1
        lo, n = start[b], start[b + 1] - start[b]
        chain = list(range(-1, n - 1)) if par is None else [int(p) for p in par[lo:lo + n]]
        rep, freq, pres = (d if t is None else float(t[b]) for t, d in ((repetition, 1.0), (frequency, 0.0), (presence, 0.0)))
        add = {}
        if bias is not None:
            for j in range(int(bias[0][b]), int(bias[0][b + 1])):
                add[int(bias[1][j])] = float(bias[2][j])
        for i in range(n + 1):
            r = lo + b + i
            z = out[r]
            count = dict(base)
            for node in path_of(chain, i):
                count[int(tok[lo + node])] = count.get(int(tok[lo + node]), 0) + 1
            for t in set(count) | prompt | set(add):
                if not 0 <= t < V:
                    continue
                c, v = count.get(t, 0), z[t]
                if c > 0 or t in prompt:
                    v = v / rep if v > 0 else v * rep
                size[r, t] = (max(size[r, t], abs(v) if np.isfinite(v) else 0.0) + abs(freq) * c + (abs(pres) if c else 0.0) +
                              abs(add.get(t, 0.0)))
                z[t] = v - freq * c - (pres if c else 0.0) + add.get(t, 0.0)
            m = -1 if words is None else r if mask_row is None else int(mask_row[r])
            if m >= 0:
                bits = (words[m][np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                z[bits == 0] = -np.inf
    return out, size


class Cache:
    """A copy of a cache (one layer) in values and 64 bits."""

    def __init__(self, cache, table):
        self.entry = [values(cache[0]), values(cache[1])]  # [pages, heads, tokens, dim]
        self.scale = [doubles(cache[2]), doubles(cache[3])]
        self.tokens = self.entry[0].shape[2]
        self.block = self.tokens // self.scale[0].shape[2]
        self.table = ints(table)

    def at(self, b, pos):
        return self.table[b, pos // self.tokens], pos % self.tokens

    def write(self, k, v, context, node_start):
        start = ints(node_start)
        for which, x in enumerate((doubles(k), doubles(v))):
            entry, scale = self.entry[which], self.scale[which]
            for b, c in enumerate(ints(context)):
                if c < 0:
                    continue
                rows = x[start[b] + b:start[b + 1] + b + 1]
                end = c + len(rows)
                for p in range(c // self.block * self.block, end, self.block):
                    page, at = self.at(b, p)
                    new = rows[max(p, c) - c:min(p + self.block, end) - c]
                    for h in range(x.shape[1]):
                        fine = np.abs(new[:, h][np.isfinite(new[:, h])])
                        most = fine.max() if fine.size else 0.0
                        need = 2.0 ** -100
                        while need * 448.0 < most:
                            need *= 2.0
                        old = scale[page, h, at // self.block]
                        size = max(old, need) if p < c else need
                        if p < c:
                            entry[page, h, at:at + c - p] *= old / size
                        f = at + max(p, c) - p
                        entry[page, h, f:f + len(new)] = np.where(np.isfinite(new[:, h]), new[:, h] / size, np.nan)
                        scale[page, h, at // self.block] = size

    def keep(self, path, accepted_len, context):
        path = ints(path)
        for which in range(2):
            entry, scale = self.entry[which], self.scale[which]
            for b, (c, n) in enumerate(zip(ints(context), ints(accepted_len))):
                if c < 0 or n <= 0:
                    continue
                first = c + 1
                for p in range(first // self.block * self.block, first + n, self.block):
                    rows = [(d, d if d < first else first + path[b, d - first]) for d in range(p, min(p + self.block, first + n))]
                    places = [self.at(b, r) for _, r in rows]
                    old = np.stack([scale[g, :, a // self.block] for g, a in places]).copy()
                    held = np.stack([entry[g, :, a] for g, a in places]).copy()
                    most = old.max(0)
                    for (d, _), o, e in zip(rows, old, held):
                        g, a = self.at(b, d)
                        entry[g, :, a] = e * (o / most)[:, None]
                    g, a = self.at(b, p)
                    scale[g, :, a // self.block] = most

    def sequence(self, b, n):
        """Keys and values of the first n positions: [heads, n, dim]."""
        got = []
        for which in range(2):
            rows = []
            for p in range(n):
                g, a = self.at(b, p)
                rows.append(self.entry[which][g, :, a] * self.scale[which][g, :, a // self.block][:, None])
            got.append(np.stack(rows, 1))
        return got

    def value_scales(self, b, n):
        """The values' scales of the first n positions: [heads, n]."""
        places = [self.at(b, p) for p in range(n)]
        return np.stack([self.scale[1][g, :, a // self.block] for g, a in places], 1)

    def attend(self, q, context, node_start, parent, scale):
        """Rows [.., query heads, dim], and the bound of what a call may be off by, entry by entry.

        A row's logits x = scale q.k are off by d: the 2 dim products are summed by the tensor core in steps of 32, each
        of which cuts off less than 2^-23 of the sum of the magnitudes for each of its products and itself; three fp32
        products with the scales (2^-24 each) and the difference to the largest x (2^-24 of the largest magnitude) follow;
        a query entry may be off by 2^-10 steps where the largest is 224 or more, 2^-17.8 of it.  The exponential is off
        by 2^-22.  A weight times its value's scale is rounded to eight bits (2^-8), or to 2^-15 where the largest such product
        of a tile (this one or one before it; with a scale of 2^-12 of some tile's largest at least, taken up to the next power
        of two) is 1 or more: 2^-14 of the largest product over all positions, with a scale of 2^-12 of the largest at least.
        The products with V are summed like those with K, in steps of 32 positions, twice.  The sum of the weights is off by 2^-24 an addition.  At last the result is rounded to bf16."""
        q = doubles(q)
        start = ints(node_start)
        par = None if parent is None else ints(parent)
        out, off = np.full(q.shape, np.nan), np.zeros(q.shape)
        group = q.shape[1] // self.entry[0].shape[1]
        for b, c in enumerate(ints(context)):
            if c < 0:
                continue
            lo, n = start[b], start[b + 1] - start[b]
            chain = list(range(-1, n - 1)) if par is None else [int(p) for p in par[lo:lo + n]]
            k, v = self.sequence(b, c + 1 + n)
            sizes = self.value_scales(b, c + 1 + n)
            for i in range(n + 1):
                seen = np.r_[np.arange(c + 1), c + 1 + np.array(sorted(path_of(chain, i)), dtype=int)]
                for h in range(q.shape[1]):
                    x, kk, vv = q[lo + b + i, h], k[h // group][seen], v[h // group][seen]
                    s = scale * (kk @ x)
                    if np.isnan(s).any() or np.isnan(vv).any():
                        continue
                    mag = abs(scale) * (np.abs(kk) @ np.abs(x))
                    d = mag * (8 * 33 + 8) * 2.0 ** -23 + 5 * 2.0 ** -24 * np.abs(s).max()
                    d = d + abs(scale) * np.abs(kk).sum(1) * np.abs(x).max() * 2.0 ** -17.8
                    w = np.exp(s - s.max())
                    p = w / w.sum()
                    o = p @ vv
                    d = np.minimum(d, 1.0)
                    size = sizes[h // group][seen]
                    lost = p * (2.0 * d + 2.0 ** -8 + 2.0 ** -21 + (len(p) / 16 + 8) * 33 * 2.0 ** -23)
                    least = 2.0 ** -14 * np.max(p * np.maximum(size, size.max() * 2.0 ** -12))
                    err = lost @ np.abs(vv) + least * (np.abs(vv) / size[:, None]).sum(0) + (p @ (2 * d) + len(p) * 2.0 ** -24) * np.abs(o)
                    out[lo + b + i, h] = o
                    off[lo + b + i, h] = err * 1.01 + (np.abs(o) + err) * 2.0 ** -8
        return out, off
