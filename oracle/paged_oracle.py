"""Plain models of the paged-cache operators (test infrastructure): page reservation with Python
loops, the e4m3 storage format from its definition, attention over gathered rows in float64.
They share no code with the CUDA path."""
from __future__ import annotations

import numpy as np

from .rtp_oracle import bf16_round, local_positions, rope_rotate

E4M3_MAX = 448.0


def e4m3_values() -> np.ndarray:
    """The value of every e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; exponent 0
    is subnormal; 0x7f and 0xff are NaN, there is no infinity."""
    out = np.zeros(256)
    for b in range(256):
        s, e, m = b >> 7, (b >> 3) & 15, b & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[b] = np.nan if (b & 0x7F) == 0x7F else (-v if s else v)
    return out


def e4m3_round(x) -> np.ndarray:
    """Nearest e4m3 value, ties to an even mantissa, values beyond +-448 to +-448."""
    x = np.asarray(x, np.float64)
    pos = e4m3_values()[:0x7F]                       # ascending, index parity = mantissa parity
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(pos, a), 1, 0x7E)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), np.nan, np.copysign(pos[pick], x))


def e4m3_rows(x):
    """Rows (last axis) as an e4m3 cache stores them: x in single precision, scale =
    max(amax / 448, 2^-126) and the quotient in single precision. Returns (values before scaling,
    scale)."""
    x = np.asarray(x, np.float64).astype(np.float32)
    scale = np.maximum(np.abs(x).max(-1) / np.float32(E4M3_MAX), np.float32(2.0 ** -126))
    return e4m3_round(x / scale[..., None]), scale


def stored_rows(x, kv: str) -> np.ndarray:
    """The values that a cache of type kv holds for rows x (float64)."""
    if kv == "bf16":
        return bf16_round(x)
    q, s = e4m3_rows(x)
    return q * s.astype(np.float64)[..., None]


def attend(q, K, V):
    """(softmax(q K^T / sqrt(d)) V, log sum exp) over the rows given; zeros and -inf for none."""
    if len(K) == 0:
        return np.zeros(V.shape[-1]), -np.inf
    z = K @ q / np.sqrt(q.shape[-1])
    m = z.max()
    w = np.exp(z - m)
    return (w @ V) / w.sum(), m + np.log(w.sum())


def positions(n: int, local: bool, sinks: int, window: int) -> np.ndarray:
    return local_positions(n, sinks, window) if local else np.arange(n)


def decode_head(q_pre, K, V, n: int, local: bool, sinks: int, window: int, base: float = 1e6):
    """One query head at position n - 1 over cache rows K, V (float64, at least n of them)."""
    if n == 0:
        return np.zeros(V.shape[-1]), -np.inf
    pos = positions(n, local, sinks, window)
    return attend(rope_rotate(q_pre, n - 1, base), K[pos], V[pos])


def reserve(page, n_pages, table, free, lens, new_lens, counters, n_new):
    """The reservation on copies of its arguments. Returns a dict of table, free, lens, counters,
    slots and error (bad arguments found on the device)."""
    table, free = np.array(table), np.array(free)
    lens, new = [int(x) for x in lens], [int(x) for x in new_lens]
    head, tail = int(counters[0]), int(counters[1])
    B, stride = table.shape
    cap = stride * page
    slots = np.full((B, n_new), -1, np.int64)
    bad = [not (0 <= a <= cap and 0 <= b <= cap) for a, b in zip(lens, new)]
    held = [0 if x else -(-a // page) for a, x in zip(lens, bad)]
    want = [0 if x else -(-b // page) for b, x in zip(new, bad)]
    returned = sum(max(h - w, 0) for h, w in zip(held, want))
    sane = 0 <= head <= tail and tail - head <= n_pages and tail - head + returned <= n_pages
    out = list(lens)
    if sane:
        avail, lacked, taken, back = tail - head, 0, 0, 0
        for b in range(B):
            if bad[b]:
                continue
            need = want[b] - held[b]
            if need > 0:
                lacked += need
                if lacked > avail:
                    continue
                for j in range(need):
                    table[b, held[b] + j] = free[(head + lacked - need + j) % n_pages]
                taken = lacked
            elif need < 0:
                for j in range(want[b], held[b]):
                    free[(tail + back) % n_pages] = table[b, j]
                    back += 1
            out[b] = new[b]
        head, tail = head + taken, tail + back
    for b in range(B):
        for j in range(n_new):
            pos = lens[b] + j
            if not bad[b] and pos < out[b]:
                slots[b, j] = int(table[b, pos // page]) * page + pos % page
    return dict(table=table, free=free, lens=np.array(out), counters=np.array([head, tail]),
                slots=slots, error=any(bad) or not sane)
