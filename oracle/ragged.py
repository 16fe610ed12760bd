"""fp64 / integer definitions of the ragged-batch operators: the plan of a
step, the 8-bit cache (scales and codes in IEEE float32, as the definition
states them; everything read from it in fp64), the attention over it, and the
adjustment of logits.  Plain numpy, one request or one row at a time.

There is no counterpart in the ByteCross pages, whose step decodes one
sequence from a bf16 cache; the definitions are those of include/bytecross.h.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 16


def pages_of(n: int) -> int:
    return -(-n // PAGE)


# ------------------------------------------------------------------ the plan
def block_tables(lens, delta, table, free_list, n_free, max_tokens):
    """Returns dict(table, free_list, n_free, lens, q_start, slots, positions)."""
    B, max_blocks = table.shape
    n_pages = len(free_list)
    cap = PAGE * max_blocks
    lens = [min(max(int(n), 0), cap) for n in lens]
    n_free = min(max(int(n_free), 0), n_pages)
    out_table, out_free = table.copy(), free_list.copy()
    pile = [int(p) for p in free_list[:n_free]]
    new_lens = list(lens)
    for b in range(B):
        if delta[b] < 0:
            new_lens[b] = max(0, lens[b] + int(delta[b]))
            pile += [int(p) for p in table[b, pages_of(new_lens[b]):pages_of(lens[b])]]
    pile = pile[:n_pages]
    room = len(pile)
    slots, positions, q_start = [], [], [0]
    asked = wanted = 0
    for b in range(B):
        n, d = lens[b], int(delta[b])
        grant = d > 0 and n + d <= cap
        if grant:
            asked += d
            grant = asked <= max_tokens
        if grant:
            need = pages_of(n + d) - pages_of(n)
            wanted += need
            grant = need == 0 or wanted <= room
        if grant:
            for i in range(need):
                out_table[b, pages_of(n) + i] = pile.pop()
            for p in range(n, n + d):
                page = int(out_table[b, p // PAGE])
                slots.append(page * PAGE + p % PAGE if 0 <= page < n_pages else -1)
                positions.append(p)
            new_lens[b] = n + d
        q_start.append(len(slots))
    for x in range(n_free, len(pile)):
        out_free[x] = pile[x]
    pad = [-1] * (max_tokens - len(slots))
    return dict(table=out_table, free_list=out_free, n_free=len(pile), lens=np.array(new_lens, np.int32),
                q_start=np.array(q_start, np.int32), slots=np.array(slots + pad, np.int32),
                positions=np.array(positions + pad, np.int32))


# ------------------------------------------------------------------ codes
CODE_MAX = {"e4m3": 448.0, "int8": 127.0}


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    mantissa bits; exponent 0 is subnormal, all ones is NaN."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m / 8.0 * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
        if e == 15 and m == 7:
            v = math.nan
        out[c] = -v if s else v
    return out


_E4M3 = e4m3_values()


def decode(codes: np.ndarray, kind: str) -> np.ndarray:
    return _E4M3[codes] if kind == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(x: np.ndarray, kind: str) -> np.ndarray:
    """Nearest code of finite values (ties to even), the largest code for
    what is beyond it."""
    x = np.asarray(x, np.float64)
    q = CODE_MAX[kind]
    x = np.clip(x, -q, q)
    if kind == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    a = np.abs(x)
    e = np.clip(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6, 8)
    m = np.rint(a / 2.0 ** (e - 3))                       # ties to even mantissas
    e, m = np.where(m == 16, e + 1, e), np.where(m == 16, 8, m)
    code = np.where(m < 8, m, (e + 7) * 8 + (m - 8)).astype(np.int64)
    return (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8)


# ------------------------------------------------------------------ the cache
def block_bytes(hd: int) -> int:
    return 2 * PAGE * hd + 32


def k_place(t: int, d: int, hd: int) -> int:
    return (d // 64) * (PAGE * 64) + t * 64 + d % 64


def v_place(t: int, d: int, hd: int) -> int:
    return PAGE * hd + (d // 4) * 64 + (t // 4) * 16 + (d % 4) * 4 + t % 4


def _places(hd):
    t, d = np.meshgrid(np.arange(PAGE), np.arange(hd), indexing="ij")
    k = (d // 64) * (PAGE * 64) + t * 64 + d % 64
    v = PAGE * hd + (d // 4) * 64 + (t // 4) * 16 + (d % 4) * 4 + t % 4
    return k, v


def scale_of(block: np.ndarray, part: int, hd: int) -> np.float32:
    at = 2 * PAGE * hd + 4 * part
    return block[at:at + 4].copy().view(np.float32)[0]


def append(pool: np.ndarray, k: np.ndarray, v: np.ndarray, slots, kind: str) -> None:
    """In place: pool uint8 [n_pages][H][block], k, v float32 [n][H][hd]."""
    n_pages, H, _ = pool.shape
    hd = k.shape[2]
    place = _places(hd)
    runs: dict[int, list[int]] = {}
    for i, s in enumerate(slots):
        if 0 <= s < n_pages * PAGE:
            runs.setdefault(int(s) // PAGE, []).append(i)
    f = np.float32
    for page, toks in runs.items():
        off = int(slots[toks[0]]) % PAGE
        for h in range(H):
            block = pool[page, h]
            for part, x in ((0, k), (1, v)):
                new = x[toks, h].astype(f)
                s_old = scale_of(block, part, hd) if off else f(0)
                m = np.abs(new).max()
                if not np.isfinite(m) or np.isnan(s_old):
                    s = f(np.nan)
                else:
                    s = f(max(s_old, max(m / f(CODE_MAX[kind]), f(2.0 ** -126)) if m > 0 else f(0)))
                inv = f(1) / s if s > 0 else f(0)
                if off and s > s_old:
                    old = decode(block[place[part][:off]], kind).astype(f)
                    block[place[part][:off]] = encode(old * s_old * inv, kind)
                if off == 0:
                    block[place[part]] = 0
                scaled = new * inv if inv > 0 else np.zeros_like(new)
                block[place[part][off:off + len(toks)]] = encode(scaled, kind)
                at = 2 * PAGE * hd + 4 * part
                block[at:at + 4] = np.array([s], f).view(np.uint8)


def read(pool: np.ndarray, slots, kind: str, hd: int):
    """fp64 keys and values [n][H][hd] of the slots (zeros outside the pool)."""
    n_pages, H, _ = pool.shape
    place = _places(hd)
    out = np.zeros((2, len(slots), H, hd))
    for i, s in enumerate(slots):
        if not 0 <= s < n_pages * PAGE:
            continue
        for h in range(H):
            block = pool[int(s) // PAGE, h]
            for part in (0, 1):
                out[part, i, h] = decode(block[place[part][int(s) % PAGE]], kind) * float(scale_of(block, part, hd))
    return out[0], out[1]


# ------------------------------------------------------------------ attention
def attention(q, pool, lens, table, kind, hd, q_start=None, max_q=1, pages=None, n_sel=None, scale=None, cap=0.0,
              window=0, slopes=None):
    """fp64 [n_q][Hq][hd]; rows of no sequence are NaN."""
    n_pages, H, _ = pool.shape
    B, max_blocks = table.shape
    Hq = q.shape[1]
    G = Hq // H
    scale = hd ** -0.5 if scale is None else scale
    place = _places(hd)
    out = np.full(q.shape, np.nan)
    for b in range(B):
        n = min(max(int(lens[b]), 0), PAGE * max_blocks)
        lo, hi = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        m = hi - lo
        if m < 1:
            continue
        for h in range(H):
            listed = range(pages_of(n)) if pages is None else \
                [int(x) for x in pages[b, h, :min(max(int(n_sel[b]), 0), pages.shape[2])] if 0 <= x < pages_of(n)]
            listed = [p for p in listed if 0 <= table[b, p] < n_pages]
            pos = np.concatenate([np.arange(p * PAGE, (p + 1) * PAGE) for p in listed]) if listed else np.zeros(0, int)
            blocks = [pool[table[b, p], h] for p in listed]
            with np.errstate(invalid="ignore"):
                kk = [decode(x[place[0]], kind) * float(scale_of(x, 0, hd)) for x in blocks]
                vv = [decode(x[place[1]], kind) * float(scale_of(x, 1, hd)) for x in blocks]
            kk = np.concatenate(kk) if kk else np.zeros((0, hd))
            vv = np.concatenate(vv) if vv else np.zeros((0, hd))
            for i in range(min(m, max_q)):
                row, p = lo + i, n - m + i
                if not 0 <= row < q.shape[0]:
                    continue
                see = (pos <= p) & (pos < n)
                if window > 0:
                    see &= pos > p - window
                for g in range(G):
                    j = h * G + g
                    if not see.any():
                        out[row, j] = 0.0
                        continue
                    x = kk[see] @ q[row, j].astype(np.float64) * scale
                    if cap > 0:
                        x = cap * np.tanh(x / cap)
                    if slopes is not None:
                        x = x - float(slopes[j]) * (p - pos[see])
                    w = np.exp(x - x.max())
                    out[row, j] = (w / w.sum()) @ vv[see]
    return out


# ------------------------------------------------------------------ logits
def logits_adjust(logits, hist=None, hist_start=None, prompt_len=None, repetition=None, frequency=None, presence=None,
                  bias_ids=None, bias_vals=None, bias_start=None, mask=None, mask_row=None):
    """fp64 [B][V]."""
    x = np.array(logits, np.float64)
    B, V = x.shape
    for b in range(B):
        if hist is not None:
            lo, hi = (min(max(int(i), 0), len(hist)) for i in hist_start[b:b + 2])
            h = [int(t) for t in hist[lo:hi]]
            pl = max(int(prompt_len[b]), 0) if prompt_len is not None else 0
            count: dict[int, int] = {}
            for t in h[pl:]:
                count[t] = count.get(t, 0) + 1
            for t in set(h):
                if not 0 <= t < V:
                    continue
                if repetition is not None:
                    r = float(repetition[b])
                    x[b, t] = x[b, t] / r if x[b, t] > 0 else x[b, t] * r
                if count.get(t):
                    x[b, t] -= (float(frequency[b]) if frequency is not None else 0.0) * count[t] + \
                        (float(presence[b]) if presence is not None else 0.0)
        if bias_ids is not None:
            lo, hi = (min(max(int(i), 0), len(bias_ids)) for i in bias_start[b:b + 2])
            add = {int(t): float(w) for t, w in zip(bias_ids[lo:hi], bias_vals[lo:hi])}
            for t, w in add.items():
                if 0 <= t < V:
                    x[b, t] += w
        if mask is not None:
            r = b if mask_row is None else int(mask_row[b])
            if 0 <= r < mask.shape[0]:
                words = mask[r].view(np.uint32)
                for t in range(V):
                    if not (int(words[t // 32]) >> (t % 32)) & 1:
                        x[b, t] = -math.inf
    return x
