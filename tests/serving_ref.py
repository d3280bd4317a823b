"""Plain references of the serving operators (step tables, rotary positions, block-scaled
8-bit caches), written from their definitions, request by request and row by row, in
Python and 64-bit numpy.  They share no code with the library."""
import math

import numpy as np
import torch

PAGE = 16
BAD_PAGE, BAD_LEN, BAD_SLOT, BAD_CHUNK, NO_PAGES = 0x1, 0x2, 0x4, 0x8, 0x20


def pages(n):
    return -(-n // PAGE)


# ------------------------------------------------------------------------- step tables

def tables(ring, state, cached, new, bt, max_tokens):
    """The definition, request by request.  Returns every output of the call."""
    ring, bt = list(ring), [list(r) for r in bt]
    N, B, MB = len(ring), len(cached), len(bt[0]) if len(bt) else 1
    head, count = state[0], state[1]
    status = 0
    ok_pool = 0 <= head < N and 0 <= count <= N
    if not ok_pool:
        head, count, status = 0, 0, BAD_PAGE
    context, starts = [], [0]
    pos, slot = [-1] * max_tokens, [-1] * max_tokens
    row, cum, alloc = 0, 0, 0
    for b in range(B):
        c, n = cached[b], new[b]
        rows = max(n, 0)
        start, row = row, row + rows
        starts.append(min(row, max_tokens))
        bad = c < 0 or c + rows > MB * PAGE or (n >= 0 and row > max_tokens)
        if bad:
            status |= BAD_LEN
        if bad or n < 0:
            context.append(0)
            continue
        need = pages(c + n) - pages(c)
        before, cum = cum, cum + need
        if need > 0 and cum > count:
            status |= NO_PAGES
            context.append(0)
            continue
        if need:
            alloc = cum
        context.append(c + n)
        for i in range(n):
            p = c + i
            pn = p // PAGE
            if pn >= pages(c):
                page = ring[(head + before + pn - pages(c)) % N]
                if not 0 <= page < N:
                    page = -1
                if p % PAGE == 0:
                    bt[b][pn] = page
            else:
                page = bt[b][pn]
            if 0 <= page < N:
                pos[start + i], slot[start + i] = p, page * PAGE + p % PAGE
            else:
                status |= BAD_PAGE
    room = N - count
    pushed = 0
    if ok_pool:
        for b in range(B):
            c = cached[b]
            if new[b] >= 0 or c < 0 or c > MB * PAGE:
                continue
            for page in bt[b][:pages(c)]:
                if page >= N:
                    status |= BAD_PAGE
                elif page >= 0:
                    if pushed < room:
                        ring[(head + count + pushed) % N] = page
                        pushed += 1
                    else:
                        status |= BAD_PAGE
    out_state = [(head + alloc) % N, count - alloc + pushed, 0, 0] if ok_pool else \
        [state[0], state[1], 0, 0]
    return dict(bt=bt, context=context, starts=starts, positions=pos, slots=slot, ring=ring,
                state=out_state, status=status)


# --------------------------------------------------------------------- rotary positions

def freqs(rd, theta=10000.0, scaling="none", factor=1.0, low=1.0, high=32.0, original_len=1):
    out = []
    for i in range(rd // 2):
        th = theta * factor ** (rd / (rd - 2)) if scaling == "base" and rd > 2 else theta
        f = th ** (-2.0 * i / rd)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            r = original_len * f / (2 * math.pi)
            g = min(1.0, max(0.0, (r - low) / (high - low)))
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return np.array(out, dtype=np.float64)


def rope(x, positions, rd, layout, f, m=1.0, transposed=False):
    """x float64 [T, H, D] turned; rows at negative positions unchanged."""
    y = np.array(x, dtype=np.float64)
    live = np.asarray(positions) >= 0
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * f * (-1.0 if transposed else 1.0)
    c, s = m * np.cos(ang), m * np.sin(ang)
    i = np.arange(rd // 2)
    ia, ib = (i, i + rd // 2) if layout == "half" else (2 * i, 2 * i + 1)
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia] = np.where(live[:, None, None], a * c - b * s, a)
    y[..., ib] = np.where(live[:, None, None], b * c + a * s, b)
    return y


# --------------------------------------------------------------- block-scaled 8-bit caches

def e4m3_values():
    """Value of every E4M3 code (bias 7, no infinity; 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = math.nan if (c & 127) == 127 else (-v if s else v)
    return out


E4M3 = e4m3_values()


def e4m3_code(x):
    """Round to the nearest E4M3 code, ties to the even one, saturating (x float64)."""
    x = np.asarray(x, dtype=np.float64)
    mag = E4M3[:127]  # ascending
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(mag, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mag[lo], mag[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return (pick | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def block_scale(top, fp8):
    if not fp8:
        return np.float32(np.float32(top) / np.float32(127.0))
    if top == 0:
        return np.float32(0)
    e = math.ceil(math.log2(float(top)) - math.log2(448.0) - 1e-9)
    while float(top) / 2.0 ** e > 448.0:
        e += 1
    while float(top) / 2.0 ** (e - 1) <= 448.0:
        e -= 1
    return np.float32(2.0 ** max(e, -126))


def block_codes(x, s, fp8):
    """x float32, s float32: the stored bytes."""
    if s == 0:
        return np.full(x.shape, 0 if fp8 else 128, dtype=np.uint8)
    q = x.astype(np.float32) / np.float32(s)
    if fp8:
        return e4m3_code(q)
    return (np.clip(np.rint(q), -127, 127) + 128).astype(np.uint8)


def block_values(byte, fp8):
    return E4M3[byte] if fp8 else byte.astype(np.float64) - 128.0


class BlockCache:
    """Bytes and scales of a block-scaled cache on the host: k [P, H, 16, D], v
    [P, H, D, 16] uint8, ks, vs [P, H] float32."""

    def __init__(self, P, H, D, fp8, fill=None, rng=None):
        self.P, self.H, self.D, self.fp8 = P, H, D, fp8
        if fill is None:
            self.k = np.zeros((P, H, PAGE, D), np.uint8)
            self.v = np.zeros((P, H, D, PAGE), np.uint8)
            self.ks = np.zeros((P, H), np.float32)
            self.vs = np.zeros((P, H), np.float32)
        else:  # anything: bytes and scales that no test may depend on
            self.k = np.full((P, H, PAGE, D), fill, np.uint8)
            self.v = np.full((P, H, D, PAGE), fill, np.uint8)
            self.ks = np.full((P, H), np.nan, np.float32)
            self.vs = np.full((P, H), np.nan, np.float32)

    def append(self, k_new, v_new, slots):
        """The definition; returns the status bits.  k_new, v_new float32 [T, H, D]."""
        status, t, T = 0, 0, len(slots)
        while t < T:
            s = int(slots[t])
            if s < 0:
                t += 1
                continue
            if s >= self.P * PAGE:
                status |= BAD_SLOT
                t += 1
                continue
            page, off = divmod(s, PAGE)
            n = 1
            while t + n < T and off + n < PAGE and int(slots[t + n]) == s + n:
                n += 1
            for x_new, store, scale, vt in ((k_new, self.k, self.ks, False), (v_new, self.v, self.vs, True)):
                for h in range(self.H):
                    blk = store[page, h].T if vt else store[page, h]  # [16, D] view
                    x = x_new[t:t + n, h]
                    need = block_scale(np.abs(x).max(), self.fp8)
                    old = scale[page, h]
                    new = need if off == 0 else max(old, need)
                    if off > 0 and new > old:
                        by = np.float32(old / new)
                        again = (block_values(blk[:off], self.fp8).astype(np.float32) * by).astype(np.float32)
                        blk[:off] = e4m3_code(again) if self.fp8 else (np.rint(again) + 128).astype(np.uint8)
                    blk[off:off + n] = block_codes(x, new, self.fp8)
                    scale[page, h] = new
            t += n
            # rows that follow in the same page out of order belong to no run
            while t < T and 0 <= int(slots[t]) < self.P * PAGE and int(slots[t]) // PAGE == page and \
                    int(slots[t - 1]) // PAGE == page and int(slots[t]) != int(slots[t - 1]) + 1:
                status |= BAD_SLOT
                t += 1
        return status

    def rows(self, h, table, L):
        """K and V of logical tokens 0 .. L-1 of kv head h, float64 [L, D]."""
        pg = np.asarray(table[:pages(L)], dtype=np.int64)
        k = block_values(self.k[pg, h], self.fp8) * self.ks[pg, h].astype(np.float64)[:, None, None]
        v = block_values(self.v[pg, h], self.fp8) * self.vs[pg, h].astype(np.float64)[:, None, None]
        return k.reshape(-1, self.D)[:L], v.transpose(0, 2, 1).reshape(-1, self.D)[:L]

    def device(self, pkv, window=0):
        t = [torch.from_numpy(a.copy()).cuda() for a in (self.k, self.v, self.ks, self.vs)]
        return pkv.KVCache(*t, window=window, kv_dtype=pkv.FP8B if self.fp8 else pkv.INT8B)

    def same_as(self, cache):
        """Whether a device cache holds these bytes and scales (NaNs alike)."""
        pairs = ((cache.k, self.k), (cache.v, self.v), (cache.k_scale, self.ks), (cache.v_scale, self.vs))
        return all(np.array_equal(a.cpu().numpy().view(np.uint8), b.view(np.uint8)) for a, b in pairs)


def attend(q, k, v, scale, first, last):
    """One row: softmax over keys first .. last in float64."""
    s = scale * (k[first:last + 1] @ q)
    p = np.exp(s - s.max())
    return (p / p.sum()) @ v[first:last + 1]


def weight(q, k, scale):
    """The largest sum of |q_i k_i| of a row's keys, as it enters exp2."""
    return float((np.abs(k) @ np.abs(q)).max()) * abs(scale) * 1.4426950408889634


def decode(bc, q, tables_, lens, scale, window=0):
    """float64 [B, Hq, D], zero rows for empty sequences; and the rows' largest weight."""
    B, Hq, D = q.shape
    out, top = np.zeros((B, Hq, D)), 0.0
    for b in range(B):
        L = int(lens[b])
        if L == 0:
            continue
        first = max(0, L - window) if window else 0
        for g in range(bc.H):
            k, v = bc.rows(g, tables_[b], L)
            for h in range(g * (Hq // bc.H), (g + 1) * (Hq // bc.H)):
                row = q[b, h].astype(np.float64)
                out[b, h] = attend(row, k, v, scale, first, L - 1)
                top = max(top, weight(row, k[first:], scale))
    return out, top


def prefill(bc, q, starts, tables_, lens, scale, window=0):
    T, Hq, D = q.shape
    out, top = np.zeros((T, Hq, D)), 0.0
    for b in range(len(lens)):
        a, e, L = int(starts[b]), int(starts[b + 1]), int(lens[b])
        for g in range(bc.H):
            k, v = bc.rows(g, tables_[b], L)
            for h in range(g * (Hq // bc.H), (g + 1) * (Hq // bc.H)):
                for t in range(a, e):
                    pos = L - (e - a) + t - a
                    first = max(0, pos - window + 1) if window else 0
                    row = q[t, h].astype(np.float64)
                    out[t, h] = attend(row, k, v, scale, first, pos)
                    top = max(top, weight(row, k[first:pos + 1], scale))
    return out, top
