"""The paged 8-bit K/V cache operators from their definitions, in numpy
float64, and inputs for their tests.  Shares no code with the library."""
import numpy as np

BLOCK = 64
NAN_CODE = 0x7F


def _e4m3_values():
    c = np.arange(256)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(e == 15) & (m == 7)] = np.nan
    return np.where(s == 1, -v, v)


E4M3 = _e4m3_values()
_POSITIVE = E4M3[:127]  # 0 .. 448, increasing


def e4m3_encode(x):
    """Nearest e4m3 code of finite or infinite x, ties to the even code, saturating."""
    a = np.abs(np.asarray(x, np.float64))
    hi = np.clip(np.searchsorted(_POSITIVE, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _POSITIVE[hi] - a, a - _POSITIVE[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(a >= 448.0, 126, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def bf16_round(x):
    """float64 -> the nearest bf16 value (ties to even), as float32."""
    b = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000
    return b.astype(np.uint32).view(np.float32)


def blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------- block tables

def extend(ctx, new, table, stack, count, T, NB):
    """(table, query_start, seq_lens, req, pos, slot, count, missing)"""
    R, MB = table.shape
    table = table.copy()
    start, req, pos, slot = [0], [], [], []
    left, missing = int(count), 0
    for r in range(R):
        c, n = max(0, int(ctx[r])), max(0, int(new[r]))
        for j in range(min(blocks(c), MB), min(blocks(c + n), MB)):
            if left > 0:
                left -= 1
                table[r, j] = stack[left]
            else:
                missing += 1
                table[r, j] = -1
        for p in range(c, c + n):
            if len(req) == T:
                break
            b = table[r, p // BLOCK] if p // BLOCK < MB else -1
            req.append(r)
            pos.append(p)
            slot.append(b * BLOCK + p % BLOCK if 0 <= b < NB else -1)
        start.append(len(req))
    pad = T - len(req)
    lens = np.minimum(np.maximum(ctx, 0).astype(np.int64) + np.maximum(new, 0), 2 ** 31 - 1)
    return (table, np.array(start), lens, np.array(req + [-1] * pad), np.array(pos + [0] * pad),
            np.array(slot + [-1] * pad), left, missing)


def release(gone, lens, table, stack, count, NB):
    """(stack, context lengths, count)"""
    stack, count = stack.copy(), int(count)
    for r in np.flatnonzero(gone):
        for b in table[r, :min(blocks(max(0, int(lens[r]))), table.shape[1])]:
            if 0 <= b < NB and count < len(stack):
                stack[count] = b
                count += 1
    return stack, np.where(gone, 0, lens), count


# ---------------------------------------------------------------- store

def _scale_for(x):
    """The smallest 2^E, E >= -100, with max |finite x| <= 448 * 2^E."""
    a = np.abs(x[np.isfinite(x)])
    amax = a.max() if a.size else 0.0
    s = 2.0 ** -100
    while amax > 448.0 * s:
        s *= 2.0
    return s


def store(x, query_start, lens, table, cache, scale):
    """x float [T, HK, D] into (cache, scale), which are copied."""
    cache, scale = cache.copy(), scale.copy()
    NB, HK = scale.shape
    for r in range(len(lens)):
        t0, t1 = int(query_start[r]), int(query_start[r + 1])
        ctx = int(lens[r]) - (t1 - t0)
        if ctx < 0:
            continue
        p = ctx
        while p < lens[r]:
            j, row = p // BLOCK, p % BLOCK
            n = min(int(lens[r]) - p, BLOCK - row)
            b = table[r, j] if j < table.shape[1] else -1
            if 0 <= b < NB:
                for h in range(HK):
                    part = x[t0 + p - ctx:t0 + p - ctx + n, h].astype(np.float64)
                    s = _scale_for(part)
                    if row:
                        s = max(s, float(scale[b, h]))
                        if s != scale[b, h]:
                            cache[b, h, :row] = e4m3_encode(E4M3[cache[b, h, :row]] * (float(scale[b, h]) / s))
                    scale[b, h] = s
                    cache[b, h, row:row + n] = e4m3_encode(np.where(np.isnan(part), 0.0, part) / s)
            p += n
    return cache, scale


# ---------------------------------------------------------------- attention

def visible(query_start, lens, r, t, window=0, prefix=None, doc=None):
    """(position, first visible key, one past the last)"""
    pos = int(lens[r]) - int(query_start[r + 1]) + t
    hi = min(int(lens[r]), max(pos + 1, int(prefix[r]) if prefix is not None else 0))
    lo = max(0, pos - window + 1 if window else 0, int(doc[t]) if doc is not None else 0)
    return pos, lo, max(lo, hi)


def attention(q, kc, vc, ks, vs, table, lens, query_start, sm_scale, window=0, softcap=0.0, slopes=None, prefix=None,
              doc=None):
    """(out, lse, tolerance of out, tolerance of lse), float64; NaN in rows of no request.

    Tolerances.  out = sum w v / sum w: the weights enter the product as two
    e4m3 terms, off by at most 2^-4 * 2^-4 of their value, or as f16, 2^-11;
    2^-7 sum w |v| / sum w covers either twice.  Small weights are rounded in
    absolute steps, but evenly to both sides: n 2^-24 max |v| of the row's
    largest weight.  Then the rounding to bf16 (half a step, 2^-8 of the
    value) and the logits' own error times the spread of v (2 dx max |v|).
    The logits: q in two e4m3 terms (off by at most 2^-18 of the row's largest
    |q|), products exact, float32 sums of 2 D = 256 terms at most: dx = sm_scale
    max|q| sum|K| (2^-18 + 2^-16)."""
    T, H, D = q.shape
    NB, HK = ks.shape
    G = H // HK
    out, lse = np.full((T, H, D), np.nan), np.full((T, H), np.nan)
    tol, ltol = np.zeros((T, H, D)), np.zeros((T, H))
    for r in range(len(lens)):
        for t in range(int(query_start[r]), int(query_start[r + 1])):
            pos, lo, hi = visible(query_start, lens, r, t, window, prefix, doc)
            j = np.arange(lo, hi)
            j = j[j // BLOCK < table.shape[1]]
            b = table[r, j // BLOCK]
            j, b = j[(b >= 0) & (b < NB)], b[(b >= 0) & (b < NB)]
            if len(j) == 0:
                out[t], lse[t] = 0.0, -np.inf
                continue
            for g in range(HK):
                K = E4M3[kc[b, g, j % BLOCK]] * ks[b, g].astype(np.float64)[:, None]
                V = E4M3[vc[b, g, j % BLOCK]] * vs[b, g].astype(np.float64)[:, None]
                h = slice(g * G, g * G + G)
                qh = q[t, h].astype(np.float64)
                x = (qh @ K.T) * sm_scale
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    x = x - slopes[h].astype(np.float64)[:, None] * np.abs(pos - j)
                m = x.max(1, keepdims=True)
                w = np.exp(x - m)
                total = w.sum(1, keepdims=True)
                out[t, h] = w @ V / total
                lse[t, h] = (m + np.log(total))[:, 0]
                dx = sm_scale * np.abs(qh).max(1, keepdims=True) * np.abs(K).sum(1).max() * (2.0 ** -18 + 2.0 ** -16)
                dx = dx + 2.0 ** -20 * (np.abs(m) + softcap + 32)
                tol[t, h] = (2.0 ** -7 * (w @ np.abs(V)) / total + len(j) * 2.0 ** -24 * np.abs(V).max() / total
                             + 2.0 ** -8 * np.abs(out[t, h]) + 2 * dx * np.abs(V).max(0))
                ltol[t, h] = dx[:, 0]
    return out, lse, tol, ltol


# ---------------------------------------------------------------- inputs

class Batch:
    """A ragged batch over a paged cache whose blocks lie in random places.
    Every position that no token sees holds NaN codes, and every block that
    none sees NaN scales."""

    def __init__(self, seed, HK, G, D, ctx, new, window=0, softcap=0.0, alibi=False, prefix=None, doc=None, pad=(0, 0),
                 spare_blocks=1, power_scales=True, q_size=1.5):
        rng = np.random.default_rng(seed)
        self.HK, self.G, self.D, self.window, self.softcap = HK, G, D, window, softcap
        R = len(ctx)
        self.lens = np.array([a + b for a, b in zip(ctx, new)], np.int32)
        self.query_start = (np.concatenate([[0], np.cumsum(new)]) + pad[0]).astype(np.int32)
        self.T = int(self.query_start[-1]) + pad[1]
        need = [blocks(int(n)) for n in self.lens]
        self.NB = sum(need) + 3
        MB = max(need + [1]) + spare_blocks
        order = rng.permutation(self.NB)
        self.table = np.full((R, MB), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        H = HK * G
        self.q = bf16_round(rng.standard_normal((self.T, H, D)) * q_size)
        self.sm_scale = float(np.float32(D ** -0.5))
        self.slopes = (2.0 ** (-8.0 * np.arange(1, H + 1) / H)).astype(np.float32) if alibi else None
        self.prefix = None if prefix is None else np.array(prefix, np.int32)
        self.doc = None if doc is None else np.concatenate(
            [np.zeros(pad[0]), np.asarray(doc), np.zeros(pad[1])]).astype(np.int32)
        seen = np.zeros((self.NB, BLOCK), bool)
        for r in range(R):
            for t in range(self.query_start[r], self.query_start[r + 1]):
                _, lo, hi = visible(self.query_start, self.lens, r, t, window, self.prefix, self.doc)
                for j in range(lo, hi):
                    seen[self.table[r, j // BLOCK], j % BLOCK] = True
        self.caches, self.scales = [], []
        for _ in range(2):
            c = e4m3_encode(rng.standard_normal((self.NB, HK, BLOCK, D)) * 110)
            c = np.where(seen[:, None, :, None], c, NAN_CODE).astype(np.uint8)
            s = 2.0 ** rng.integers(-8, -5, (self.NB, HK))
            if not power_scales:
                s = s * rng.uniform(0.5, 2.0, s.shape)
            s = np.where(seen.any(1)[:, None], s, np.nan).astype(np.float32)
            self.caches.append(c)
            self.scales.append(s)

    def expected(self):
        return attention(self.q, *self.caches, *self.scales, self.table, self.lens, self.query_start, self.sm_scale,
                         self.window, self.softcap, self.slopes, self.prefix, self.doc)
