"""Plain 64-bit statements of the calls in include/pa_serving.h (numpy, CPU), and
the small pools that their tests share."""
from __future__ import annotations

from fractions import Fraction

import numpy as np
import torch

BS = 16


def f64(t):
    """A tensor's values in 64 bits."""
    return t.detach().cpu().to(torch.float64).numpy()


def tables_for(lens, mbs, g, extra=0):
    """Shuffled block tables (-1 behind each sequence's blocks) and the number
    of blocks they use; ``extra``: blocks of each sequence beyond those."""
    t = torch.full((len(lens), mbs), -1, dtype=torch.int32)
    n = [(int(x) + BS - 1) // BS + extra for x in lens]
    perm = torch.randperm(sum(n), generator=g).to(torch.int32)
    c = 0
    for b, k in enumerate(n):
        t[b, :k] = perm[c:c + k]
        c += k
    return t, max(1, sum(n))


def e4m3_pool(g, shape):
    """Codes and page scales of normal values, as the quantiser makes them."""
    x = torch.randn(shape, generator=g) * torch.rand(shape[0], shape[1], 1, 1, generator=g).mul(3).add(.1)
    s = x.abs().amax((2, 3)) / torch.tensor(448.)
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def rope(x, positions, inv_freq, axis, adjacent, amplitude=1.0):
    """x [T][H][D] (64 bits), positions [axes][T]."""
    y = x.copy()
    half = len(inv_freq)
    for i in range(half):
        a = positions[axis[i]].astype(np.float64) * inv_freq[i]
        c, s = amplitude * np.cos(a)[:, None], amplitude * np.sin(a)[:, None]
        lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[:, :, lo] = x[:, :, lo] * c - x[:, :, hi] * s
        y[:, :, hi] = x[:, :, hi] * c + x[:, :, lo] * s
    return y


def inverse_two_pi(bits=320):
    """1 / 2 pi as a Fraction, to about 2^-bits (Machin: pi / 4 = 4 atan 1/5 - atan 1/239)."""
    def atan(n):
        term = (1 << bits) // n
        total, k = term, 3
        while term:
            term //= -n * n
            total += term // k
            k += 2
        return total
    return Fraction(1 << bits, 8 * (4 * atan(5) - atan(239)))


def rope_angles(positions, inv_freq):
    """positions [T] times inv_freq [pairs] (doubles, as given), reduced to one turn without
    rounding and then to 64 bits: radians [T][pairs]."""
    turn = inverse_two_pi()
    out = np.empty((len(positions), len(inv_freq)))
    for i, f in enumerate(inv_freq):
        step = Fraction(float(f)) * turn
        for t, p in enumerate(positions):
            out[t, i] = 2 * np.pi * float((int(p) * step + Fraction(1, 2)) % 1 - Fraction(1, 2))
    return out


def keys(k_cache, k_scale, table, h, L):
    blocks = table[:(L + BS - 1) // BS].long()
    k = k_cache[blocks, h]
    if k_cache.dtype == torch.uint8:
        k = f64(k.view(torch.float8_e4m3fn).float()) * f64(k_scale[blocks, h])[:, None, None]
    else:
        k = f64(k)
    return k.reshape(-1, k.shape[-1])[:L]


def attention_weights(w, q, k_cache, k_scale, tables, lens, scale, decay, fresh):
    """Returns (the weights, their tolerance): see the derivation below.

    A logit is a sum of D products, exact in fp32 one by one, accumulated in
    fp32 in D/16 <= 8 steps of 16 (each step's alignment may drop up to 2^-22 of
    the largest partial sum), then multiplied by the page scale and the softmax
    scale (2^-24 each): |error| <= 8 * 2^-22 S + 2^-22 |s| with S = scale * sum
    |q_i k_i|.  The weight p = 2^(s - m) / l takes the error of its own logit
    and, through l, the largest of the row's; ex2.approx adds 2^-22 relative to p
    and to each term of l, the sums over partitions and rows and the division
    under 2^-20 together; the old weight times decay 2^-23.  A weight below
    2^-126 may be flushed to zero."""
    out, tol = w.copy(), np.zeros_like(w)
    B, n_q, Hq, D = q.shape
    Hkv = w.shape[1]
    G = Hq // Hkv
    for b in range(B):
        L = int(lens[b])
        for h in range(Hkv):
            if L == 0:
                continue
            k = keys(k_cache, k_scale, tables[b], h, L)
            got, off = np.zeros(L), np.zeros(L)
            for i in range(n_q):
                n = L - n_q + 1 + i
                if n <= 0:
                    continue
                for g in range(G):
                    x = q[b, i, h * G + g]
                    s = scale * (k[:n] @ x)
                    e = np.exp(s - s.max())
                    p = e / e.sum()
                    S = scale * (np.abs(k[:n]) @ np.abs(x))
                    err = 2. ** -19 * S + 2. ** -22 * np.abs(s)
                    got[:n] += p
                    off[:n] += p * (err + err.max() + 2. ** -19) + 2. ** -125
            old = decay * w[b, h, :L] if decay else np.zeros(L)
            old = np.where(np.arange(L) < L - fresh, old, 0.)
            out[b, h, :L] = old + got
            tol[b, h, :L] = off + 2. ** -22 * np.abs(out[b, h, :L])
    return out, tol


def evict_choice(w, L, keep, first, recent):
    """The kept positions of one (sequence, kv head), in order."""
    if L <= keep:
        return np.arange(L)
    mid = np.arange(first, L - recent)
    key = np.where(np.isnan(w[mid]), -np.inf, w[mid])
    # a NaN is lower than everything, -inf included
    order = sorted(range(len(mid)), key=lambda i: (np.isnan(w[mid[i]]), -key[i], mid[i]))
    heavy = mid[sorted(order[:keep - first - recent])]
    return np.concatenate([np.arange(first), heavy, np.arange(L - recent, L)]).astype(np.int64)


def evict(pools, scales, w, tables, lens, spare, keep, first, recent):
    """pools, scales: lists of CPU tensors (K, V), changed in place.  Returns
    (new_lens, kept lists, tables_out)."""
    B, Hkv = w.shape[:2]
    new, kept = np.minimum(lens, keep), {}
    out = torch.full_like(spare, -1)
    src_pools = [p.clone() for p in pools]
    src_scales = [None if s is None else s.clone() for s in scales]
    for b in range(B):
        L = int(lens[b])
        n = min(tables.shape[1], spare.shape[1])
        if L > keep:
            out[b] = spare[b]
        else:
            out[b, :n] = tables[b, :n]
        for h in range(Hkv):
            at = evict_choice(w[b, h], L, keep, first, recent)
            kept[b, h] = at
            if L <= keep:
                continue
            at = torch.from_numpy(at)
            blk = tables[b, at // BS].long()
            for pool, sc, src, ssc in zip(pools, scales, src_pools, src_scales):
                rows = src[blk, h, at % BS]
                for page in range((keep + BS - 1) // BS):
                    d = int(spare[b, page])
                    r = rows[page * BS:(page + 1) * BS]
                    if sc is None:
                        pool[d, h, :len(r)] = r
                        continue
                    x = r.view(torch.float8_e4m3fn).float() * ssc[blk[page * BS:(page + 1) * BS], h][:, None]
                    amax = x.abs().max()
                    s = amax / torch.tensor(448.) if amax > 0 else torch.tensor(1.)
                    sc[d, h] = s
                    pool[d, h, :len(r)] = (x / s).to(torch.float8_e4m3fn).view(torch.uint8)
    return new, kept, out


def verify(p, q, x, u, n_b, n):
    """One sequence: p [n + 1][V], q [n][V] or None, all 64 bits; (tokens, accepted)."""
    clean = lambda a: np.clip(np.nan_to_num(a, nan=0., posinf=2.), 0., 2.)  # noqa: E731
    V = p.shape[1]
    r = 0
    while r < n_b:
        if not 0 <= x[r] < V:
            break
        qx = 1. if q is None else clean(q[r, x[r]])
        if not u[r] * qx < clean(p[r, x[r]]):
            break
        r += 1
    w = clean(p[r])
    if r < n_b:
        if q is None:
            qr = np.zeros(V)
            if 0 <= x[r] < V:
                qr[x[r]] = 1
        else:
            qr = clean(q[r])
        left = np.maximum(w - qr, 0)
        if left.sum() > 0:
            w = left
    cdf = np.cumsum(w)
    tok = -1 if cdf[-1] == 0 else int(np.searchsorted(cdf, u[n] * cdf[-1], side="right"))
    return [int(t) for t in x[:r]] + [tok] + [-1] * (n - r), r
