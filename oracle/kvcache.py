"""Oracle of the paged key / value cache: rotary positions, page tables and
attention in plain numpy, 64 bits, written from the definitions in
``include/kvcache.h`` and sharing no code with the kernels."""
from __future__ import annotations

import math

import numpy as np


# ---- element types -------------------------------------------------------------

def to_f64(bits: np.ndarray, dtype: str) -> np.ndarray:
    """Values of an array that holds a type's bits (u16 for f16 and bf16)."""
    if dtype == "bf16":
        return (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return bits.view({"f16": np.float16, "f32": np.float32}[dtype]).astype(np.float64)


def half_step(dtype: str) -> float:
    """The largest relative error of one rounding to the type."""
    return {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]


# ---- rotary positions ------------------------------------------------------------

def rope_thetas(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, slow=1.0, fast=32.0):
    out = []
    for j in range(rot // 2):
        b = base
        if scaling == "base" and rot > 2:
            b = base * factor ** (rot / (rot - 2))
        theta = b ** (-2.0 * j / rot)
        if scaling == "linear":
            theta /= factor
        elif scaling == "ramp":
            turns = original_len * theta / (2 * math.pi)
            w = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            theta = theta * w + theta / factor * (1.0 - w)
        out.append(theta)
    return out


def rope(x, pos, thetas, layout="half", magnitude=1.0, inverse=False):
    """x [tokens, heads, dim] (float64) rotated; also the sum of the absolute
    terms behind each element, which rounding errors scale with."""
    y, size = x.copy(), np.abs(x)
    half = len(thetas)
    for t in range(x.shape[0]):
        for j, theta in enumerate(thetas):
            # whole turns are taken out of the product exactly; the product itself is rounded to 64 bits, off by 2^-53 of it
            angle = math.fmod(float(pos[t]) * theta, 2 * math.pi)
            c, s = magnitude * math.cos(angle), magnitude * math.sin(-angle if inverse else angle)
            a, b = (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + half)
            u, v = x[t, :, a], x[t, :, b]
            y[t, :, a], y[t, :, b] = u * c - v * s, u * s + v * c
            size[t, :, a] = size[t, :, b] = abs(magnitude) * (np.abs(u) + np.abs(v))
    return y, size


# ---- page tables -------------------------------------------------------------------

class Pages:
    """Tables, lengths, counts and pools (arrays [pages, ...]) of a cache."""

    def __init__(self, table, lens, refs, slots, pools=()):
        self.table, self.lens, self.refs = table.copy(), lens.copy(), refs.copy()
        self.slots, self.pools = slots, [p.copy() for p in pools]

    def _free(self):
        return [p for p in range(len(self.refs)) if self.refs[p] <= 0]

    def _row_ok(self, r):
        return 0 <= r < len(self.table) and 0 <= self.lens[r] <= self.slots * self.table.shape[1]

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.table):
                continue
            for c in range(self.table.shape[1]):
                p = self.table[r, c]
                if p != -1 and 0 <= p < len(self.refs):
                    self.refs[p] -= 1
                self.table[r, c] = -1
            self.lens[r] = 0

    def extend(self, rows, add):
        free, total, ok = self._free(), 0, []
        start = self.lens.copy()
        for r, n in zip(rows, add):
            good = self._row_ok(r) and n >= 0 and start[r] + n <= self.slots * self.table.shape[1]
            first = -(-int(start[r]) // self.slots) if good else 0
            end = -(-int(start[r] + n) // self.slots) if good else 0
            total += end - first
            good = good and total <= len(free)
            ok.append(int(good))
            if good:
                for k in range(first, end):
                    p = free[total - (end - k)]
                    self.table[r, k], self.refs[p] = p, 1
                self.lens[r] = start[r] + n
        return ok

    def fork(self, src, dst):
        free, total, ok = self._free(), 0, []
        start = self.lens.copy()
        for s, d in zip(src, dst):
            good = self._row_ok(s) and 0 <= d < len(self.table) and start[d] == 0
            tail = good and start[s] % self.slots != 0
            total += int(tail)
            good = good and total <= len(free)
            ok.append(int(good))
            if not good:
                continue
            full = int(start[s]) // self.slots
            self.table[d, :] = -1
            for c in range(full):
                p = self.table[s, c]
                self.table[d, c] = p
                self.refs[p] += 1
            if tail:
                p = free[total - 1]
                self.table[d, full], self.refs[p] = p, 1
                for pool in self.pools:
                    pool[p] = pool[self.table[s, full]]
            self.lens[d] = start[s]
        return ok

    def compact(self):
        n = len(self.refs)
        used = int((self.refs > 0).sum())
        holes = [p for p in range(used) if self.refs[p] <= 0]
        moves = [p for p in range(used, n) if self.refs[p] > 0]
        place = {p: p for p in range(used)}
        for h, m in zip(holes, moves):
            place[m] = h
            self.refs[h], self.refs[m] = self.refs[m], 0
            for pool in self.pools:
                pool[h] = pool[m]
        for r in range(self.table.shape[0]):
            for c in range(self.table.shape[1]):
                p = int(self.table[r, c])
                if 0 <= p < n:
                    self.table[r, c] = place.get(p, -1)
        return used


# ---- attention -----------------------------------------------------------------------

def attention(q, k_pool, v_pool, table, lens, slots, prefix_row, prefix_len, rows, scale):
    """q [batch, q_len, heads, dim], pools [pages, slots, kv heads, dim], all
    float64.  Returns o, lse, the weighted sum of |v| behind each element of o,
    the largest sum of |q . k| terms behind a score, and how many keys a query
    sees."""
    batch, q_len, heads, dim = q.shape
    kv = k_pool.shape[2]
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    weight, score_size = np.zeros(q.shape), np.zeros(q.shape[:3])
    seen = np.zeros(q.shape[:3], dtype=np.int64)
    for b in range(batch):
        row = rows[b] if rows is not None else b
        for j in range(q_len):
            keys = [(prefix_row, t) for t in range(prefix_len)]
            keys += [(row, t) for t in range(max(0, int(lens[row]) - q_len + 1 + j))]
            if not keys:
                continue
            page = np.array([table[r][t // slots] for r, t in keys])
            slot = np.array([t % slots for _, t in keys])
            for h in range(heads):
                g = h // (heads // kv)
                k, v = k_pool[page, slot, g], v_pool[page, slot, g]
                s = scale * (k @ q[b, j, h])
                m = s.max()
                w = np.exp(s - m)
                o[b, j, h] = w @ v / w.sum()
                weight[b, j, h] = w @ np.abs(v) / w.sum()
                lse[b, j, h] = m + math.log(w.sum())
                score_size[b, j, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, j, h])).max()
                seen[b, j, h] = len(keys)
    return o, lse, weight, score_size, seen


def attention_by_head(q, k_pool, v_pool, table, lens, slots, prefix_row, prefix_len, rows, scale):
    """attention() for long prefixes: a head's queries meet the prefix in one
    product, and each sequence's own tokens behind it."""
    batch, q_len, heads, dim = q.shape
    group = heads // k_pool.shape[2]
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    weight, score_size = np.zeros(q.shape), np.zeros(q.shape[:3])
    seen = np.zeros(q.shape[:3], dtype=np.int64)

    def keys(row, n, g):
        t = np.arange(n)
        page, slot = np.asarray(table[row])[t // slots], t % slots
        return k_pool[page, slot, g], v_pool[page, slot, g]

    for h in range(heads):
        k0, v0 = keys(prefix_row, prefix_len, h // group)
        shared = scale * (q[:, :, h] @ k0.T)
        size = np.zeros((batch, q_len))
        if prefix_len:
            size = abs(scale) * (np.abs(q[:, :, h]) @ np.abs(k0).T).max(-1)
        for b in range(batch):
            row = rows[b] if rows is not None else b
            k1, v1 = keys(row, int(lens[row]), h // group)
            for j in range(q_len):
                n = max(0, int(lens[row]) - q_len + 1 + j)
                if prefix_len + n == 0:
                    continue
                s = np.concatenate((shared[b, j], scale * (k1[:n] @ q[b, j, h])))
                m = s.max()
                w = np.exp(s - m)
                w0, w1, total = w[:prefix_len], w[prefix_len:], w.sum()
                o[b, j, h] = (w0 @ v0 + w1 @ v1[:n]) / total
                weight[b, j, h] = (w0 @ np.abs(v0) + w1 @ np.abs(v1[:n])) / total
                lse[b, j, h] = m + math.log(total)
                own = abs(scale) * (np.abs(k1[:n]) @ np.abs(q[b, j, h])).max(initial=0.0)
                score_size[b, j, h] = max(size[b, j], own)
                seen[b, j, h] = prefix_len + n
    return o, lse, weight, score_size, seen
