"""Pages, the layout of a packed batch and attention over a prompt, from their definitions on the CPU
(numpy; attention in 64 bits).  Shares no code with the library."""
import numpy as np


def reserve(table, held, free, num_free, tokens, page, num_pages):
    """sfx_pages_reserve on copies: (table, held, free, num_free, missing)."""
    table, held, free = table.copy(), held.copy(), free.copy()
    B, width = table.shape
    nf = min(max(int(num_free), 0), num_pages)
    need = [-(-max(int(t), 0) // page) for t in tokens]
    held = np.clip(held, 0, width)
    released = []
    for b in range(B):
        for j in range(need[b], held[b]):
            released.append(int(table[b, j]))
            table[b, j] = -1
    room = nf + len(released)
    wanted, missing, taken = 0, np.zeros(B, np.int32), []
    new = held.copy()
    for b in range(B):
        if need[b] <= held[b]:
            new[b] = need[b]
            continue
        e = need[b] - int(held[b])
        if need[b] > width:
            missing[b] = e
            continue
        wanted += e
        if wanted > room:
            missing[b] = e
            continue
        taken += [(b, j) for j in range(held[b], need[b])]
        new[b] = need[b]
    for a, (b, j) in enumerate(taken):
        if a < len(released):
            table[b, j] = released[a]
        else:
            nf -= 1
            table[b, j] = free[nf]
    for p in released[len(taken):]:
        free[nf] = p
        nf += 1
    return table, new.astype(np.int32), free, nf, missing


def layout(table, start, count, N, page, num_pages):
    """sfx_step_layout: offsets, seq_lens, request, position, slots."""
    B, width = table.shape
    off = [0]
    for c in count:
        off.append(min(off[-1] + max(int(c), 0), N))
    seq = np.zeros(B, np.int64)
    req, pos, slot = (np.full(N, -1, np.int64) for _ in range(3))
    for b in range(B):
        a = max(int(start[b]), 0)
        n = off[b + 1] - off[b]
        seq[b] = a + n
        for t in range(n):
            i, p = off[b] + t, a + t
            req[i], pos[i] = b, p
            if p // page < width and 0 <= table[b, p // page] < num_pages:
                slot[i] = int(table[b, p // page]) * page + p % page
    return np.array(off), seq, req, pos, slot


def prompt(q, k, v, scale, window, sinks):
    """One request: q [n, Hq, d], k, v [n, H, d] float64.  (out, sum of p |v|, largest sum |q||k| *
    scale) per row; infinities and NaN count where they are seen and nowhere else."""
    n, Hq, d = q.shape
    G = Hq // k.shape[1]
    out, mag, dots = np.zeros((n, Hq, d)), np.zeros((n, Hq, d)), np.zeros((n, Hq))
    j = np.arange(n)
    for t in range(n):
        see = j <= t
        if window:
            see &= (j > t - window) | (j < sinks)
        for h in range(Hq):
            kk, vv = k[see, h // G], v[see, h // G]
            s = kk @ q[t, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            with np.errstate(invalid="ignore"):
                out[t, h] = w @ vv
                mag[t, h] = w @ np.abs(vv)
            dots[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
    return out, mag, dots
