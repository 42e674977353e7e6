"""Plain 64-bit statements of the calls in include/pa_request.h (numpy, CPU)."""
from __future__ import annotations

from collections import deque

import numpy as np
import torch

from _serving_ref import BS, f64


def rows_of(cache, scale, table, h, L, num_blocks):
    """Keys or values [L][D] of one sequence and kv head in 64 bits, and which of them are there
    (their block id is a valid one)."""
    D = cache.shape[-1]
    x, ok = np.zeros((L, D)), np.zeros(L, dtype=bool)
    for j in range(0, L, BS):
        p = int(table[j // BS])
        if 0 <= p < num_blocks:
            r = cache[p, h, :min(BS, L - j)]
            x[j:j + BS] = f64(r.view(torch.float8_e4m3fn).float()) * float(scale[p, h]) \
                if cache.dtype == torch.uint8 else f64(r)
            ok[j:j + BS] = True
    return x, ok


def prefill(out, q, kc, vc, ks, vs, tables, lens, starts, max_context, scale, window):
    """out [T][Hq][D] (64 bits) with the rows that have a result replaced; also, for each
    element, sum_j p_j |V_j| and max_j |s_j| of its row, from which tolerances are made."""
    out = out.copy()
    mass, big = np.zeros_like(out), np.zeros_like(out)
    T, Hq, D = out.shape
    NB, Hkv = kc.shape[:2]
    G = Hq // Hkv
    for b in range(len(lens)):
        a, e = int(starts[b]), int(starts[b + 1])
        if not 0 <= a <= e <= T:
            continue
        L, n = int(lens[b]), e - a
        out[a:e] = 0
        if not 0 <= L <= max_context:
            continue
        for h in range(Hkv):
            k, ok = rows_of(kc, ks, tables[b], h, L, NB)
            v, _ = rows_of(vc, vs, tables[b], h, L, NB)
            for i in range(n):
                pos = L - n + i
                see = ok[:max(pos + 1, 0)].copy()
                if window:
                    see[:max(0, pos - window + 1)] = False
                if pos < 0 or not see.any():
                    continue
                j = np.flatnonzero(see)
                x = q[a + i, h * G:(h + 1) * G]
                s = scale * (x @ k[j].T)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                at = np.s_[a + i, h * G:(h + 1) * G]
                out[at] = p @ v[j]
                mass[at] = p @ np.abs(v[j])
                # what the products of a logit add up to, whatever their signs
                big[at] = (abs(scale) * (np.abs(x) @ np.abs(k[j]).T)).max(-1, keepdims=True)
    return out, mass, big


def prefill_tol(ref, mass, big, half_step, p_half_step):
    """Each weight is rounded to the products' type (p_half_step of it) after an error of
    its exponent: a logit's products are exact in fp32 and added in at most 8 steps that
    may each lose 2^-22 of the sum of their sizes S; scale, page scale and the base-2 factor
    round by 2^-24 each; so a weight is off by 2 (2^-19 S + 2^-20) with its normaliser's
    share, and the exponential by 2^-21.  The products with V and their sums over partitions
    add 2^-18 of the mass; the result is rounded once (16-bit results have a smallest step)."""
    weight = p_half_step + 2. ** -18 * big + 2. ** -17
    return half_step * (np.abs(ref) + weight * mass) + weight * mass + 2. ** -24


class Pages:
    """The pool's pages by reference counts, on the host."""

    def __init__(self, tables, held, ref):
        self.tables, self.held, self.ref = (np.array(x.tolist(), dtype=np.int64) for x in (tables, held, ref))

    def free_pages(self):
        return deque(np.flatnonzero(self.ref <= 0).tolist())

    def alloc(self, rows, lens):
        free, granted, out = self.free_pages(), [], False
        for r, L in zip(rows, lens):
            want = -(-int(L) // BS)
            if not 0 <= r < len(self.held) or not 0 <= self.held[r] <= self.tables.shape[1] or \
                    L < 0 or want > self.tables.shape[1]:
                granted.append(0)
                continue
            need = max(0, want - int(self.held[r]))
            out = out or need > len(free)
            granted.append(0 if out else 1)
            for _ in range(0 if out else need):
                p = free.popleft()
                self.tables[r, self.held[r]] = p
                self.held[r] += 1
                self.ref[p] = 1
        return granted

    def free(self, rows):
        for r in rows:
            if not 0 <= r < len(self.held) or not 0 <= self.held[r] <= self.tables.shape[1]:
                continue
            for j in range(self.held[r]):
                p = self.tables[r, j]
                if 0 <= p < len(self.ref) and self.ref[p] > 0:
                    self.ref[p] -= 1
                self.tables[r, j] = -1
            self.held[r] = 0

    def fork(self, src, dst, lens, pools):
        """lens is changed in place; pools: tensors with one entry a page."""
        free, granted, out = self.free_pages(), [], False
        for a, c in zip(src, dst):
            if not (0 <= a < len(self.held) and 0 <= c < len(self.held)) or a == c or \
                    not 0 <= self.held[a] <= self.tables.shape[1] or \
                    not 0 <= lens[a] <= self.held[a] * BS:
                granted.append(0)
                continue
            L = int(lens[a])
            out = out or (L % BS > 0 and not free)
            granted.append(0 if out else 1)
            if out:
                continue
            full = L // BS
            self.tables[c, :full] = self.tables[a, :full]
            for p in self.tables[a, :full]:
                if 0 <= p < len(self.ref):
                    self.ref[p] += 1
            if L % BS:
                p, old = free.popleft(), int(self.tables[a, full])
                self.tables[c, full] = p
                self.ref[p] = 1
                if 0 <= old < len(self.ref):
                    for x in pools:
                        x[p] = x[old]
            self.held[c] = -(-L // BS)
            lens[c] = L
        return granted

    def compact(self, pools):
        """Returns (moved_to, number of live pages)."""
        live = int((self.ref > 0).sum())
        to = np.where(self.ref > 0, np.arange(len(self.ref)), -1)
        holes = deque(p for p in range(live) if self.ref[p] <= 0)
        for p in range(live, len(self.ref)):
            if self.ref[p] > 0:
                h = holes.popleft()
                to[p] = h
                for x in pools:
                    x[h] = x[p]
                self.ref[h], self.ref[p] = self.ref[p], 0
        for r in range(len(self.held)):
            if not 0 <= self.held[r] <= self.tables.shape[1]:
                continue
            for j in range(self.held[r]):
                p = self.tables[r, j]
                if 0 <= p < len(self.ref):
                    self.tables[r, j] = to[p]
        return to, live


def logits(x, spec, b, i):
    """One row [V] in 64 bits; spec: dict of numpy arrays (None for what is left out).
    Returns (the adjusted row, the sum of the sizes of what was added up)."""
    V = len(x)
    x = x.copy()
    history = np.zeros(0, dtype=np.int64)
    P = 0
    if spec["history"] is not None:
        L = int(spec["history_lens"][b])
        if 0 <= L <= spec["history"].shape[1]:
            history = spec["history"][b, :L].astype(np.int64)
        P = 0 if spec["prompt_lens"] is None else min(max(int(spec["prompt_lens"][b]), 0), len(history))
    drafts = np.zeros(0, dtype=np.int64) if spec["draft_tokens"] is None else \
        spec["draft_tokens"][b, :i].astype(np.int64)
    good = lambda t: t[(t >= 0) & (t < V)]  # noqa: E731
    count = np.bincount(good(np.concatenate([history[P:], drafts])), minlength=V)
    seen = (count > 0) | (np.bincount(good(history[:P]), minlength=V) > 0)
    par = lambda n, v: v if spec[n] is None else float(spec[n][b])  # noqa: E731
    r, f, p = par("repetition", 1.), par("frequency", 0.), par("presence", 0.)
    x[seen] = np.where(x[seen] > 0, x[seen] / r, x[seen] * r)
    size = np.abs(x)
    hit = count > 0
    x[hit] -= f * count[hit] + p
    size[hit] += np.abs(f) * count[hit] + np.abs(p)
    if spec["bias_tokens"] is not None:
        for t, v in zip(spec["bias_tokens"][b], spec["bias_values"][b]):
            if 0 <= t < V:
                x[t] += v
                size[t] += abs(v)
    if spec["allowed"] is not None:
        bits = np.unpackbits(spec["allowed"][b, i].view(np.uint8), bitorder="little")[:V]
        x[bits == 0] = -np.inf
    return x, size


def probabilities(x, temp):
    x = np.where(np.isnan(x), -np.inf, x)
    p = np.zeros_like(x)
    m = x.max()
    if m == -np.inf:
        return p
    if not temp > 0:
        p[int(np.flatnonzero(x == m)[0])] = 1
        return p
    if m == np.inf:
        p[x == m] = 1
    else:
        d = x - m
        p = np.exp(np.where(np.isinf(d), -np.inf, np.where(np.isinf(d), 0, d) / temp))
    return p / p.sum()
