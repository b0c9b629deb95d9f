"""The 8-bit KV cache, the attention over it and the draft verification, from their definitions
in 64 bits on the CPU (numpy).  Shares no code with the library."""
import numpy as np

E_LO, E_HI, BLOCK = -32, 31, 32


def e4m3_values():
    """The 256 values of e4m3: sign, four exponent bits (bias 7), three of the fraction; the
    last magnitude is NaN."""
    v = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[b] = -x if b > 127 else x
    v[127] = v[255] = np.nan
    return v


VALUES = e4m3_values()
_POS = VALUES[:127]
_MID = (_POS[1:] + _POS[:-1]) / 2


def encode(x):
    """Codes of float64 values: nearest, ties to the even code, saturating; NaN to NaN."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    lo = np.searchsorted(_MID, a, side="left")    # a tie stays on the lower code
    hi = np.searchsorted(_MID, a, side="right")   # ... or goes to the upper one
    c = np.where(lo % 2 == 0, lo, hi).astype(np.uint8)
    c = np.where(np.isnan(x), np.uint8(127), c)
    return np.where(np.signbit(x), c | 128, c).astype(np.uint8)


def needed(amax):
    """Least e in range with amax <= 448 * 2^e."""
    e = E_LO
    while e < E_HI and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


class Cache:
    """codes [pages, heads, page, dim] per tensor and exponents [pages, heads, page / 32]."""

    def __init__(self, pages, page, heads, dim):
        self.shape = (pages, heads, page, dim)
        self.page = page
        self.code = {n: np.zeros(self.shape, np.uint8) for n in "kv"}
        self.exp = {n: np.full((pages, heads, page // BLOCK), E_LO) for n in "kv"}

    def pack(self, name):
        """The library's layout of one tensor (uint8) and its scales (float32)."""
        P, H, page, d = self.shape
        c = self.code[name]
        scale = (2.0 ** self.exp[name]).astype(np.float32)
        if name == "k":
            return c.reshape(P, H, page, d // 64, 64).transpose(0, 1, 3, 2, 4).copy(), scale
        out = np.zeros((P, H, page // 32, d // 32, 16, 4, 2, 2, 4), np.uint8)
        for tok in range(32):
            j, g, i = tok // 16, tok % 16 // 4, tok % 4
            x = c.reshape(P, H, page // 32, 32, d // 32, 16, 2)[:, :, :, tok]
            out[:, :, :, :, :, g, :, j, i] = x
        return out, scale

    def values(self, name, table, upto):
        """[upto, heads, dim] float64 values of one request's tokens; NaN-free `mapped` mask."""
        P, H, page, d = self.shape
        out, ok = np.zeros((upto, H, d)), np.zeros(upto, bool)
        for p in range(0, upto, BLOCK):
            pid = table[p // page] if p // page < len(table) else -1
            if pid < 0 or pid >= P:
                continue
            n = min(BLOCK, upto - p)
            o = p % page
            out[p:p + n] = VALUES[self.code[name][pid, :, o:o + n]].transpose(1, 0, 2) * \
                (2.0 ** self.exp[name][pid, :, o // BLOCK])[None, :, None]
            ok[p:p + n] = True
        return out, ok

    def write(self, name, x, table, start, count):
        """x [T, heads, dim] float64, as sfx_kv_write."""
        P, H, page, d = self.shape
        count = min(count, x.shape[0])
        if start < 0 or count <= 0:
            return
        for blk in range(start // BLOCK, (start + count - 1) // BLOCK + 1):
            pi = blk * BLOCK // page
            pid = table[pi] if pi < len(table) else -1
            if pid < 0 or pid >= P:
                continue
            o = blk * BLOCK % page
            lo, hi = max(start, blk * BLOCK), min(start + count, (blk + 1) * BLOCK)
            for h in range(H):
                new = x[lo - start:hi - start, h]
                fin = np.abs(new[np.isfinite(new)])
                e = needed(fin.max() if fin.size else 0.0)
                code = self.code[name][pid, h, o:o + BLOCK]
                if blk * BLOCK < start:
                    old = int(self.exp[name][pid, h, o // BLOCK])
                    e = max(e, old)
                    if e != old:
                        n = start - blk * BLOCK
                        code[:n] = encode(VALUES[code[:n]] * 2.0 ** (old - e))
                code[lo - blk * BLOCK:hi - blk * BLOCK] = encode(new * 2.0 ** -e)
                self.exp[name][pid, h, o // BLOCK] = e


def attention(cache, q, table, seq_len, q_len, scale, window, sinks):
    """q [T, heads_q, dim] float64: (out, sum of p |v|, largest sum |q||k| * scale) per row."""
    T, Hq, d = q.shape
    H = cache.shape[1]
    G = Hq // H
    cap = len(table) * cache.page
    L, n = min(max(seq_len, 0), cap), min(max(q_len, 0), T)
    out, mag, dots = np.zeros((T, Hq, d)), np.zeros((T, Hq, d)), np.zeros((T, Hq))
    if L == 0:
        return out, mag, dots
    k, ok = cache.values("k", table, L)
    v, _ = cache.values("v", table, L)
    j = np.arange(L)
    for t in range(n):
        p = L - n + t
        see = (j <= p) & ok
        if window:
            see &= (j > p - window) | (j < sinks)
        if not see.any():
            continue
        for h in range(Hq):
            kk, vv = k[see, h // G], v[see, h // G]
            s = kk @ q[t, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[t, h] = w @ vv
            mag[t, h] = w @ np.abs(vv)
            dots[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
    return out, mag, dots


def verify(logits, draft, nv, ua, us, temp):
    """One request: logits [k + 1, V] float64.  Returns (sampled [k + 1], accepted)."""
    k1, V = logits.shape
    nv = min(max(nv, 0), k1 - 1)
    x = np.where(np.isnan(logits), -np.inf, logits)
    out = np.full(k1, -1, np.int32)

    def weights(row):
        m = row.max()
        if m == -np.inf:
            return None
        if m == np.inf:
            return (row == np.inf).astype(np.float64)
        with np.errstate(over="ignore", under="ignore"):
            e = (row - m) / np.float64(temp) if temp != np.inf else np.where(
                row == -np.inf, -np.inf, 0.0)
            return np.exp(e)

    greedy = not temp > 0
    for i in range(nv + 1):
        d = int(draft[i]) if i < nv else -1
        valid = 0 <= d < V
        if greedy:
            best = int(np.argmax(x[i])) if x[i].max() > -np.inf else -1
            if valid and best == d:
                out[i] = d
                continue
            out[i] = best
            return out, i
        w = weights(x[i])
        if w is not None and valid and float(ua[i]) * w.sum() < w[d]:
            out[i] = d
            continue
        if w is None:
            return out, i
        if valid:
            w = w.copy()
            w[d] = 0.0
        c = np.cumsum(w)
        if c[-1] <= 0:
            out[i] = int(np.argmax(x[i]))
            return out, i
        j = int(np.searchsorted(c, float(us) * c[-1], side="right"))
        out[i] = j if j < V else int(np.nonzero(w)[0][-1])
        return out, i
    return out, nv
