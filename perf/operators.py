"""Measured cases of the verification step's operators: the 8-bit KV cache's write and read, the
attention over it, and the verification of a draft.

The cache's layout (elements of one page and head):
  k        [pages, heads, dim/64, page, 64]              e4m3 codes, token-major in 64-dim slabs
  v        [pages, heads, page/32, dim/32, 16, 4, 2, 2, 4]  e4m3 codes; indices r, g, f, j, i hold
           token 16 j + 4 g + i of the 32-token block and dim 32 (slab) + 2 r + f
  k_scale, v_scale  [pages, heads, page/32]  float32 powers of two; a value is code * scale
Block scale: the least 2^e with amax <= 448 * 2^e, e within [-32, 31] (-32 for an all-zero block).
"""
import math

import torch

own = False

E_LO, E_HI = -32, 31
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sampled token a request, a small engine: the call's latency counts
        dict(name="write-append-B4-T1", op="write", B=4, T=1, lo=1, hi=500, heads=4, dim=64,
             page=32, type="fp16"),
        # a draft of 16 and the sampled token for a full decode batch
        dict(name="write-draft-B256-T17", op="write", B=256, T=17, lo=100, hi=1000, heads=8,
             dim=128, page=64, type="bf16"),
        # prompts written in one go
        dict(name="write-prompt-B8-T8192", op="write", B=8, T=8192, lo=0, hi=0, heads=8, dim=128,
             page=64, type="bf16"),
        # a short prefix read back
        dict(name="read-B4-T333", op="read", B=4, T=333, heads=4, dim=64, page=32, type="fp16"),
        # long prefixes read back to be moved to another engine
        dict(name="read-B8-T16384", op="read", B=8, T=16384, heads=8, dim=128, page=64,
             type="bf16"),
        # plain decoding of a small batch: the smallest call
        dict(name="attend-B4-S512-T1", op="attend", B=4, T=1, lo=128, hi=512, heads=4, group=2,
             dim=64, page=32, window=0, sinks=0, type="fp16"),
        # plain decoding, one token a request, ordinary lengths
        dict(name="attend-B64-S4096-T1", op="attend", B=64, T=1, lo=1024, hi=4096, heads=8,
             group=4, dim=128, page=64, window=0, sinks=0, type="bf16"),
        # a draft of 16 verified over long contexts: the ordinary call of the step, at its largest
        dict(name="attend-B32-S16384-T17", op="attend", B=32, T=17, lo=8192, hi=16384, heads=8,
             group=4, dim=128, page=64, window=0, sinks=0, type="bf16"),
        # one long request alone on the card
        dict(name="attend-B1-S32768-T17", op="attend", B=1, T=17, lo=32768, hi=32768, heads=8,
             group=8, dim=128, page=128, window=0, sinks=0, type="bf16"),
        # a layer with a sliding window and four first tokens that stay visible
        dict(name="attend-window-B64-S16384-T9", op="attend", B=64, T=9, lo=4096, hi=16384,
             heads=8, group=4, dim=128, page=64, window=2048, sinks=4, type="bf16"),
        # a small vocabulary and batch: latency
        dict(name="verify-B4-k8-V1024", op="verify", B=4, k=8, V=1024, take=0.7, greedy=False,
             type="fp32"),
        # a full decode batch over a large vocabulary
        dict(name="verify-B256-k16-V151936", op="verify", B=256, k=16, V=151936, take=0.8,
             greedy=False, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "verify", "verify"])
    if op == "verify":
        while True:
            c = dict(op=op, B=_log(rng, 1, 256), k=rng.randint(1, 32), V=_log(rng, 1000, 152000),
                     take=round(rng.uniform(0.3, 0.95), 3), greedy=rng.random() < 0.2,
                     type=rng.choice(["bf16", "fp16", "fp32"]))
            if c["B"] * (c["k"] + 1) * c["V"] * SIZE[c["type"]] <= 1.3e9:
                return c
    heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 256])
    page = rng.choice([32, 64, 96, 128, 256])
    if op == "write":
        while True:
            t = _log(rng, 1, 8192)
            c = dict(op=op, B=_log(rng, 1, 256), T=t, lo=0, hi=rng.choice([0, 1000]), heads=heads,
                     dim=dim, page=page, type=rng.choice(["bf16", "fp16", "fp32"]))
            if c["B"] * t * heads * dim <= 6e7 and c["B"] * (t + c["hi"]) * heads * dim <= 3e8:
                return c
    if op == "read":
        while True:
            c = dict(op=op, B=_log(rng, 1, 64), T=_log(rng, 1, 16384), heads=heads, dim=dim,
                     page=page, type=rng.choice(["bf16", "fp16", "fp32"]))
            if c["B"] * c["T"] * heads * dim * SIZE[c["type"]] <= 2.6e8:
                return c
    while True:
        hi = _log(rng, 1, 32768)
        win = rng.choice([0, 0, _log(rng, 1, 4096)])
        c = dict(op=op, B=_log(rng, 1, 64), T=rng.choice([1, 1, rng.randint(2, 33)]),
                 lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, heads=heads,
                 group=rng.choice([1, 2, 4, 5, 7, 8, 16]), dim=dim, page=page, window=win,
                 sinks=rng.choice([0, 1, 4]) if win else 0, type=rng.choice(["bf16", "fp16"]))
        if c["B"] * hi * heads * dim <= 5e8 and \
                c["B"] * hi * heads * dim * c["group"] * c["T"] <= 3e10:
            return c


# ------------------------------------------------------------------ the cache's format
def _pow2(e):
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    f, x = torch.frexp(amax)
    e = torch.where(f <= 0.875, x - 9, x - 8).clamp(E_LO, E_HI)
    return torch.where(amax > 0, e, torch.full_like(e, E_LO))


def _code(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _pack_k(c, page):  # [n, heads, page, dim] -> the layout of k
    n, h, _, d = c.shape
    return c.view(n, h, page, d // 64, 64).permute(0, 1, 3, 2, 4)


def _unpack_k(c):  # the layout of k, pages gathered to [..., heads, dim/64, page, 64]
    x = c.movedim(-3, -2)
    return x.reshape(*x.shape[:-2], -1)


def _pack_v(c, page):
    n, h, _, d = c.shape
    x = c.view(n, h, page // 32, 2, 4, 4, d // 32, 16, 2)  # b, j, g, i, slab, r, f
    return x.permute(0, 1, 2, 6, 7, 4, 8, 3, 5)


def _unpack_v(c):  # [..., page/32, dim/32, 16, 4, 2, 2, 4] -> [..., page, dim]
    n = c.dim() - 7
    x = c.permute(*range(n), n, n + 5, n + 3, n + 6, n + 1, n + 2, n + 4)
    return x.reshape(*x.shape[:n], x.shape[n] * 32, -1)


def _kv(g, shape, dev):
    """Keys or values as projections give them: normal, some channels larger, tokens of other
    sizes among them."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= torch.exp(0.7 * torch.randn(shape[-1], generator=g, device=dev))
    x *= torch.exp(0.4 * torch.randn(shape[:-1] + (1,), generator=g, device=dev))
    return x


def _cache(g, pages, heads, dim, page, dev):
    """A filled cache; made in slices to bound the memory."""
    out = {"k": torch.empty((pages, heads, dim // 64, page, 64), dtype=torch.uint8, device=dev),
           "v": torch.empty((pages, heads, page // 32, dim // 32, 16, 4, 2, 2, 4),
                            dtype=torch.uint8, device=dev),
           "k_scale": torch.empty((pages, heads, page // 32), device=dev),
           "v_scale": torch.empty((pages, heads, page // 32), device=dev)}
    step = max(1, (1 << 27) // (heads * dim * page))
    for name, pack in (("k", _pack_k), ("v", _pack_v)):
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = _kv(g, (n, heads, page, dim), dev)
            e = _exponent(x.view(n, heads, page // 32, 32, dim).abs().amax((-1, -2)))
            c = _code(x.view(n, heads, page // 32, 32, dim) * _pow2(-e)[..., None, None])
            c = c.view(torch.uint8).view(n, heads, page, dim)
            out[name][p:p + n] = pack(c, page)
            out[name + "_scale"][p:p + n] = _pow2(e)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def ints(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=g, device=dev, dtype=torch.int32)

    op, B = case["op"], case["B"]
    s = {"op": op, "case": dict(case)}
    t = TYPES[case["type"]]
    if op == "verify":
        k, V, a = case["k"], case["V"], case["take"]
        # the target gives the drafted token the probability `take`; one in 1 - take of the
        # drafted tokens is one that the target finds unlikely
        x = torch.empty((B, k + 1, V), dtype=t, device=dev)
        temp = 0.5 + torch.rand((B,), generator=g, device=dev)
        greedy = torch.rand((B,), generator=g, device=dev) < (1.0 if case["greedy"] else 0.125)
        draft = torch.randint(0, V, (B, k), generator=g, device=dev, dtype=torch.int32)
        for b in range(0, B, 8):
            x[b:b + 8] = (2.0 * torch.randn((min(8, B - b), k + 1, V), generator=g, device=dev)
                          * temp[b:b + 8, None, None])
        top = (math.log(a / (1 - a)) + math.log(V) + 2.0) * temp
        likely = torch.rand((B, k), generator=g, device=dev) < a
        at = torch.where(likely, draft, torch.randint(0, V, (B, k), generator=g, device=dev,
                                                      dtype=torch.int32)).long()
        x[:, :k].scatter_(2, at[:, :, None], top[:, None, None].expand(B, k, 1).to(t))
        s.update(logits=x, draft=draft, num_valid=ints(max(1, k - 3), k, B),
                 u_accept=torch.rand((B, k), generator=g, device=dev),
                 u_sample=torch.rand((B,), generator=g, device=dev),
                 temperature=torch.where(greedy, torch.zeros_like(temp), temp))
        return s
    heads, dim, page, T = case["heads"], case["dim"], case["page"], case["T"]
    hi = {"write": case.get("hi", 0) + T, "read": T + 64, "attend": case.get("hi", 0)}[op]
    width = hi // page + 4
    s["page_table"] = torch.randperm(B * width, generator=g, device=dev).to(torch.int32).view(
        B, width)
    s.update(_cache(g, B * width, heads, dim, page, dev))
    if op == "write":
        s["new_k"] = _kv(g, (B, T, heads, dim), dev).to(t)
        s["new_v"] = _kv(g, (B, T, heads, dim), dev).to(t)
        s["start"] = ints(case["lo"], case["hi"], B)
        s["count"] = ints(max(1, T - T // 8), T, B)
    elif op == "read":
        s["start"] = ints(0, 63, B)
        s["count"] = ints(max(1, T - T // 8), T, B)
    else:
        s["q"] = torch.randn((B, T, heads * case["group"], dim), generator=g, device=dev).to(t)
        s["seq_lens"] = ints(case["lo"], case["hi"], B)
        s["q_lens"] = ints(max(1, T - 2), T, B)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"write": _write, "read": _read, "attend": _attend, "verify": _verify}[s["op"]](s)


def _own(s):
    import suffix_match_drafter_amd as sfx

    op, case = s["op"], s["case"]
    if op == "verify":
        return sfx.verify(s["logits"], s["draft"], s["num_valid"], s["u_accept"], s["u_sample"],
                          s["temperature"])
    if "cache" not in s:  # the handle over the cache's buffers
        s["cache"] = sfx.KVCache(s["k"].shape[0], case["page"], case["heads"], case["dim"],
                                 buffers=(s["k"], s["v"], s["k_scale"], s["v_scale"]))
    if op == "write":
        s["cache"].write(s["new_k"], s["new_v"], s["page_table"], s["start"], s["count"])
        return _cache_out(s)
    if op == "read":
        return s["cache"].read(s["page_table"], s["start"], s["count"], case["T"],
                               TYPES[case["type"]])
    return s["cache"].attend(s["q"], s["page_table"], s["seq_lens"], s["q_lens"],
                             window=case["window"], sinks=case["sinks"])


def _cache_out(s):
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _write(s):
    """The new tokens' blocks, 32 tokens by 32, old tokens of a block carried to its new scale."""
    case, new_t = s["case"], s["case"]["T"]
    B, page, dev = case["B"], case["page"], s["k"].device
    nb = (new_t + 30) // 32 + 1
    start, count = s["start"].long(), s["count"].long()
    blk = start[:, None] // 32 + torch.arange(nb, device=dev)                  # [B, nb]
    pg = torch.gather(s["page_table"].long(), 1,
                      (blk * 32 // page).clamp(max=s["page_table"].shape[1] - 1))
    sub = blk % (page // 32)
    pos = blk[:, :, None] * 32 + torch.arange(32, device=dev)                  # [B, nb, 32]
    src = pos - start[:, None, None]
    new = (src >= 0) & (src < count[:, None, None])
    old = src < 0
    touched = new.any(2)
    src = src.clamp(0, new_t - 1)
    rows = torch.arange(B, device=dev)[:, None, None]
    heads, dim = case["heads"], case["dim"]
    k6 = s["k"].view(-1, heads, dim // 64, page // 32, 32, 64)
    for name, x in (("k", s["new_k"]), ("v", s["new_v"])):
        x = x[rows, src].float().permute(0, 1, 3, 2, 4)                        # B nb h 32 d
        n = new[:, :, None, :, None]
        if name == "k":
            c = k6[pg, :, :, sub]                                              # B nb h d/64 32 64
            c = _unpack_k(c)
        else:
            c = _unpack_v(s["v"][pg, :, sub].unsqueeze(3)).reshape(B, nb, heads, 32, dim)
        scale = s[name + "_scale"]
        s_old = scale[pg, :, sub]                                              # B nb h
        e = _exponent((x.abs() * n).amax((-1, -2)))
        s_new = torch.where(old[:, :, 0, None], torch.maximum(_pow2(e), s_old), _pow2(e))
        s_new = torch.where(touched[:, :, None], s_new, s_old)
        v_old = c.contiguous().view(torch.float8_e4m3fn).float()
        moved = _code(v_old * (s_old / s_new)[..., None, None])
        keep = (old & touched[:, :, None])[:, :, None, :, None]
        out = torch.where(n, _code(x / s_new[..., None, None]).view(torch.uint8),
                          torch.where(keep, moved.view(torch.uint8), c))
        if name == "k":
            k6[pg, :, :, sub] = out.reshape(B, nb, heads, 32, dim // 64, 64).transpose(3, 4)
        else:
            s["v"][pg, :, sub] = _pack_v(out.reshape(B * nb, heads, 32, dim), 32).reshape(
                B, nb, heads, dim // 32, 16, 4, 2, 2, 4)
        scale[pg, :, sub] = s_new
    return _cache_out(s)


def _tokens(s):
    """All tokens of each request's pages in float32: [B, heads, tokens, dim] twice."""
    pt = s["page_table"].long()
    got = []
    for name, unpack in (("k", _unpack_k), ("v", _unpack_v)):
        x = unpack(s[name][pt])                                                # B n h page d
        x = x.contiguous().view(torch.float8_e4m3fn).float()
        B, n, h, page, d = x.shape
        x = x.view(B, n, h, page // 32, 32, d) * s[name + "_scale"][pt][..., None, None]
        got.append(x.view(B, n, h, page, d).transpose(1, 2).reshape(B, h, n * page, d))
    return got


def _read(s):
    T = s["case"]["T"]
    j = torch.arange(T, device=s["k"].device)
    at = (s["start"].long()[:, None] + j)[:, None, :, None]
    live = (j < s["count"][:, None])[:, None, :, None]
    t, got = TYPES[s["case"]["type"]], []
    for x in _tokens(s):
        at_x = at.expand(-1, x.shape[1], -1, x.shape[3])
        x = torch.where(live, torch.gather(x, 2, at_x), torch.zeros((), device=x.device))
        got.append(x.to(t).transpose(1, 2).contiguous())
    return tuple(got)


def _attend(s):
    case = s["case"]
    B, T, h, G, d = case["B"], case["T"], case["heads"], case["group"], case["dim"]
    k, v = _tokens(s)
    S = k.shape[2]
    j = torch.arange(S, device=k.device)
    t = torch.arange(T, device=k.device)
    pos = (s["seq_lens"] - s["q_lens"])[:, None] + t                           # [B, T]
    pos = torch.where(t < s["q_lens"][:, None], pos, torch.full_like(pos, -1))
    see = j <= pos[:, :, None]
    if case["window"]:
        see &= (j > pos[:, :, None] - case["window"]) | (j < case["sinks"])
    q = s["q"].float().view(B, T, h, G, d).permute(0, 2, 1, 3, 4).reshape(B * h, T * G, d)
    x = torch.bmm(q, k.view(B * h, S, d).transpose(1, 2)).view(B, h, T, G, S) / math.sqrt(d)
    x = x.masked_fill(~see[:, None, :, None], -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    z = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(B * h, T * G, S), v.view(B * h, S, d)).view(B, h, T, G, d)
    o = torch.where(z > 0, o / z, torch.zeros((), device=o.device))
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, h * G, d).to(s["q"].dtype)


def _verify(s):
    """In 64 bits: the tests `u Z < w` and the place of `u Z` in the running sum sit next to
    borders."""
    B, k1, V = s["logits"].shape
    k, dev = k1 - 1, s["logits"].device
    temp = s["temperature"].double()
    greedy = ~(temp > 0)
    x = s["logits"].double()
    top = x.amax(2, keepdim=True)
    v = torch.arange(V, device=dev, dtype=torch.int32)
    best = torch.where(x == top, v, torch.full_like(v, V)).amin(2)             # lowest index
    w = torch.exp((x - top) / torch.where(greedy, 1.0, temp)[:, None, None])
    z = w.sum(2)
    d = s["draft"].long()
    wd = torch.gather(w[:, :k], 2, d[:, :, None])[:, :, 0]
    ok = torch.where(greedy[:, None], best[:, :k] == d, s["u_accept"].double() * z[:, :k] < wd)
    ok &= torch.arange(k, device=dev) < s["num_valid"][:, None]
    n = ok.to(torch.int64).cumprod(1).sum(1)                                   # accepted
    rows = torch.arange(B, device=dev)
    w = w[rows, n]                                                             # [B, V]
    out = torch.gather(torch.cat([d, torch.zeros_like(d[:, :1])], 1), 1, n[:, None])
    rejected = (n < s["num_valid"])[:, None]
    w = torch.where(rejected & (v == out), torch.zeros_like(w), w)
    c = w.cumsum(1)
    token = (c <= s["u_sample"].double()[:, None] * c[:, -1:]).sum(1).clamp(max=V - 1)
    token = torch.where(greedy, best[rows, n].long(), token)
    i = torch.arange(k1, device=dev)
    full = torch.cat([d, d[:, :1]], 1)
    sampled = torch.where(i < n[:, None], full,
                          torch.where(i == n[:, None], token[:, None], -torch.ones_like(full)))
    return sampled.to(torch.int32), n.to(torch.int32)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, B, es = case["op"], case["B"], SIZE[case["type"]]
    if op == "verify":
        # rows up to the first rejected draft: a drafted token is accepted with about take^2
        a, nv = case["take"] ** 2, max(1, case["k"] - 1.5)
        rows = (1 - a ** (nv + 1)) / (1 - a)
        return {"bytes": B * rows * case["V"] * es, "flops": 4 * B * rows * case["V"]}
    heads, dim, T = case["heads"], case["dim"], case["T"]
    tok = 2 * heads * dim
    mean_t = (max(1, T - T // 8) + T) / 2
    if op in ("write", "read"):
        return {"bytes": B * mean_t * tok * (1 + es), "flops": 2 * B * mean_t * tok}
    seen = (case["lo"] + case["hi"]) / 2
    if case["window"]:
        seen = min(seen, case["window"] + T - 1 + case["sinks"])
    rows = T * case["group"] * heads * dim
    per_row = min(seen, case["window"] + case["sinks"]) if case["window"] else seen
    return {"bytes": B * (seen * tok + 2 * rows * es), "flops": 4 * B * rows * per_row}


# ------------------------------------------------------------------ the definition in 64 bits
def _two(e):
    """2^e, exactly (a device's pow need not be)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _value_of_byte(dev):
    """The 256 values of e4m3: sign, four exponent bits with bias 7, three of the fraction."""
    b = torch.arange(256, device=dev)
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _two(e - 10))
    mag = torch.where((b & 127) == 127, torch.full_like(mag, math.nan), mag)
    return torch.where(b > 127, -mag, mag)


def _nearest(x):
    """x rounded to e4m3's values, ties to even, in 64 bits."""
    x = x.clamp(-448.0, 448.0)
    step = _two(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x / step) * step


def _at(s, b, pos):
    """Request b's codes' values and scales at token positions `pos`, [n, heads, dim] each."""
    page, heads, dim = s["case"]["page"], s["case"]["heads"], s["case"]["dim"]
    tab = _value_of_byte(pos.device)
    p = s["page_table"][b].long()[pos // page]
    o = pos % page
    d = torch.arange(dim, device=pos.device)
    h = torch.arange(heads, device=pos.device)
    P, H, D = p[:, None, None], h[None, :, None], d[None, None, :]
    O = o[:, None, None]
    u = O % 32
    ik = (P, H, D // 64, O, D % 64)
    iv = (P, H, O // 32, D // 32, D % 32 // 2, u % 16 // 4, D % 2, u // 16, u % 4)
    sc = (p[:, None], h[None], (o // 32)[:, None])
    return {"k": (ik, tab[s["k"][ik].long()], s["k_scale"][sc].double()),
            "v": (iv, tab[s["v"][iv].long()], s["v_scale"][sc].double()), "scale_at": sc}


def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["B"]
    if op == "verify":
        return None  # whole numbers
    dev = s["k"].device
    if op == "write":
        tab = _value_of_byte(dev)
        out = {"k": tab[s["k"].long()], "v": tab[s["v"].long()],
               "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
        for b in range(B):
            a, n = int(s["start"][b]), int(s["count"][b])
            first = a // 32 * 32
            got = _at(s, b, torch.arange(first, a + n, device=dev))
            for name in "kv":
                idx, val, sc = got[name]
                val = val * sc[:, :, None]
                fresh = s["new_" + name][b, :n].double()
                val[a - first:] = fresh
                m = torch.full(((len(val) + 31) // 32 * 32, case["heads"]), 0.0, device=dev,
                               dtype=torch.float64)
                m[a - first:len(val)] = fresh.abs().amax(2)
                m = m.view(-1, 32, case["heads"]).amax(1)
                e = torch.ceil(torch.log2(m.clamp(min=2.0 ** -80) / 448)).clamp(E_LO, E_HI)
                if a > first:
                    e[0] = torch.maximum(e[0], torch.log2(sc[0]))
                full = _two(e).repeat_interleave(32, 0)[:len(val)]
                out[name][idx] = _nearest(val / full[:, :, None])
                out[name + "_scale"][got["scale_at"]] = full
        return out
    if op == "read":
        zero = torch.zeros((B, case["T"], case["heads"], case["dim"]), dtype=torch.float64,
                           device=dev)
        out = (zero, zero.clone())
        for b in range(B):
            n = int(s["count"][b])
            got = _at(s, b, int(s["start"][b]) + torch.arange(n, device=dev))
            for o, name in zip(out, "kv"):
                o[b, :n] = got[name][1] * got[name][2][:, :, None]
        return out
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    for b in range(B):
        L, n = int(s["seq_lens"][b]), int(s["q_lens"][b])
        if L == 0 or n == 0:
            continue
        at = torch.arange(L, device=dev)
        got = _at(s, b, at)
        k, v = (got[x][1] * got[x][2][:, :, None] for x in "kv")               # [L, heads, dim]
        for h in range(case["heads"]):
            kh, vh = k[:, h].contiguous(), v[:, h].contiguous()
            q = s["q"][b, :n, h * case["group"]:(h + 1) * case["group"]].double()
            x = (q.reshape(-1, case["dim"]) @ kh.t()).view(n, case["group"], L)
            x = x / math.sqrt(case["dim"])
            pos = L - n + torch.arange(n, device=dev)[:, None]
            see = at <= pos
            if case["window"]:
                see = see & ((at > pos - case["window"]) | (at < case["sinks"]))
            x = torch.where(see[:, None], x, torch.full_like(x, -math.inf))
            p = torch.softmax(x, -1).nan_to_num(0.0)
            o = p.reshape(-1, L) @ vh
            out[b, :n, h * case["group"]:(h + 1) * case["group"]] = o.view(n, -1, case["dim"])
    return out
