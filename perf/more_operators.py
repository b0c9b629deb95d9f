"""Measured cases of continuous batching around the verification step: pages handed out on the device,
the layout of a packed batch, the 8-bit cache's write by slots, attention of whole prompts and attention
of packed chunks, drafts and single tokens over the cache.

A packed batch holds the requests' rows one behind the other; `offsets` [B + 1] says where each starts.
The cache's layout (elements of one page and head):
  k        [pages, heads, dim/64, page, 64]              e4m3 codes, token-major in 64-dim slabs
  v        [pages, heads, page/32, dim/32, 16, 4, 2, 2, 4]  e4m3 codes; indices r, g, f, j, i hold
           token 16 j + 4 g + i of the 32-token block and dim 32 (slab) + 2 r + f
  k_scale, v_scale  [pages, heads, page/32]  float32 powers of two; a value is code * scale
Block scale: the least 2^e with amax <= 448 * 2^e, e within [-32, 31] (-32 for an all-zero block).
"""
import math
import random

import torch

own = False

E_LO, E_HI = -32, 31
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a small engine's decode batch takes a page now and then: the call's latency counts
        dict(name="reserve-B32", op="reserve", B=32, lo=1, hi=2000, swap=0.0, grow=17, page=64,
             spare=1.2),
        # a large one: a quarter of the requests ends, others of up to 16384 tokens come in, and
        # the pages do not last for all of them
        dict(name="reserve-B1024-admit", op="reserve", B=1024, lo=100, hi=16384, swap=0.25,
             grow=17, page=32, spare=1.0),
        # 64 drafts of 16 and the sampled token
        dict(name="layout-B64-T17", op="layout", B=64, lo=17, hi=17, at=4000, page=64, pad=0),
        # a full batch with prompts among it, padded to a fixed number of rows
        dict(name="layout-B256-N20000", op="layout", B=256, lo=1, hi=150, at=8000, page=64,
             pad=672),
        # drafts of 16 and the sampled token written by slots
        dict(name="slots-B64-T17", op="slots", B=64, lo=1, hi=33, at=2000, heads=8, dim=128,
             page=64, type="bf16"),
        # prompts of up to 4096 tokens written by slots
        dict(name="slots-B8-T4096", op="slots", B=8, lo=512, hi=4096, at=0, heads=8, dim=128,
             page=64, type="bf16"),
        # a few short prompts of a small model
        dict(name="prompt-B4-S200", op="prompt", B=4, lo=10, hi=200, heads=4, group=2, dim=64,
             window=0, sinks=0, type="fp16"),
        # a batch of ordinary prompts, packed
        dict(name="prompt-B16-S2048", op="prompt", B=16, lo=128, hi=2048, heads=8, group=4,
             dim=128, window=0, sinks=0, type="bf16"),
        # long prompts
        dict(name="prompt-B2-S8192", op="prompt", B=2, lo=8192, hi=8192, heads=8, group=4,
             dim=128, window=0, sinks=0, type="bf16"),
        # a small engine's step: drafts and single tokens, a layer with a window and first tokens
        dict(name="chunk-small-window", op="chunk", chunks=1, T=64, drafts=7, rows=9, lo=64,
             hi=600, heads=4, group=2, dim=64, page=32, window=128, sinks=4, type="fp16"),
        # chunks of two prompts beside 32 drafts: the step of a server under load
        dict(name="chunk-2x1024-32x17", op="chunk", chunks=2, T=1024, drafts=32, rows=17, lo=2048,
             hi=8192, heads=8, group=4, dim=128, page=64, window=0, sinks=0, type="bf16"),
        # the last chunk of one long prompt
        dict(name="chunk-1x2048-S32768", op="chunk", chunks=1, T=2048, drafts=0, rows=1, lo=32768,
             hi=32768, heads=8, group=4, dim=128, page=64, window=0, sinks=0, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["reserve", "layout", "slots", "prompt", "prompt", "chunk", "chunk"])
    page = rng.choice([32, 64, 96, 128, 256])
    if op == "reserve":
        hi = _log(rng, 16, 16384)
        return dict(op=op, B=_log(rng, 1, 1024), lo=rng.randint(1, hi), hi=hi,
                    swap=rng.choice([0.0, 0.1, 0.5]), grow=rng.randint(1, 33), page=page,
                    spare=rng.choice([1.0, 1.1, 2.0]))
    if op == "layout":
        while True:
            hi = _log(rng, 1, 2000)
            c = dict(op=op, B=_log(rng, 1, 512), lo=rng.randint(0, hi), hi=hi,
                     at=_log(rng, 1, 16384), page=page, pad=rng.choice([0, rng.randint(1, 300)]))
            if c["B"] * hi <= 20000:
                return c
    heads, dim = rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128, 128, 256])
    if op == "slots":
        while True:
            hi = _log(rng, 1, 4096)
            c = dict(op=op, B=_log(rng, 1, 256), lo=rng.randint(1, hi), hi=hi,
                     at=rng.choice([0, _log(rng, 1, 2000)]), heads=heads, dim=dim, page=page,
                     type=rng.choice(["bf16", "fp16", "fp32"]))
            if c["B"] * hi * heads * dim <= 4e7 and c["B"] * (hi + c["at"]) * heads * dim <= 2e8:
                return c
    group, win = rng.choice([1, 2, 4, 5, 7, 8, 16]), rng.choice([0, 0, _log(rng, 1, 4096)])
    rest = dict(heads=heads, group=group, dim=dim, window=win,
                sinks=rng.choice([0, 1, 4, 70]) if win else 0, type=rng.choice(["bf16", "fp16"]))
    if op == "prompt":
        while True:
            hi = _log(rng, 1, 8192)
            c = dict(op=op, B=_log(rng, 1, 64), lo=rng.randint(1, hi), hi=hi, **rest)
            if c["B"] * hi * hi * heads * group * dim <= 2.7e11 and \
                    c["B"] * hi * heads * group * dim <= 1.5e8:
                return c
    while True:
        hi = _log(rng, 32, 32768)
        t = min(hi, _log(rng, 1, 4096))
        c = dict(op=op, chunks=rng.randint(0, 3), T=t, drafts=rng.choice([0, _log(rng, 1, 64)]),
                 rows=rng.choice([1, rng.randint(2, 32)]), lo=rng.randint(max(t, 32), max(hi, 32)),
                 hi=hi, page=page, **rest)
        n = c["chunks"] + c["drafts"]
        pairs = (c["chunks"] * t + c["drafts"] * c["rows"]) * hi * heads * group * dim
        if n and pairs <= 2.6e11 and n * hi * heads * dim <= 5e8:
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


def _place(slot, heads, dim, page):
    """Indices of the codes of tokens at slots [n], in k and in v: [n, heads, dim] each."""
    p, o = (slot // page)[:, None, None], (slot % page)[:, None, None]
    h = torch.arange(heads, device=slot.device)[None, :, None]
    d = torch.arange(dim, device=slot.device)[None, None, :]
    u = o % 32
    return ((p, h, d // 64, o, d % 64),
            (p, h, o // 32, d // 32, d % 32 // 2, u % 16 // 4, d % 2, u // 16, u % 4))


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
            out[name][p:p + n] = pack(c.view(torch.uint8).view(n, heads, page, dim), page)
            out[name + "_scale"][p:p + n] = _pow2(e)
    return out


# ------------------------------------------------------------------ inputs
def _spread(rng, n, lo, hi):
    """n whole numbers in [lo, hi] whose sum does not depend on rng (pairs around the middle)."""
    a = [rng.randint(lo, hi) for _ in range(n // 2)]
    x = a + [lo + hi - v for v in a] + [(lo + hi) // 2] * (n % 2)
    rng.shuffle(x)
    return x


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _running(x):
    out = [0]
    for v in x:
        out.append(out[-1] + v)
    return out


def _ragged(s, lens, start, dev):
    """What a step's program knows of its packed rows: offsets, and each row's request and place."""
    off = _running(lens)
    s["lens"], s["first"] = lens, off
    s["offsets"] = _i32(off, dev)
    s["request"] = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], device=dev)
    s["row"] = torch.arange(off[-1], device=dev) - s["offsets"].long()[s["request"]]
    s["position"] = s["row"] + _i32(start, dev).long()[s["request"]]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rng = random.Random(seed)
    op = case["op"]
    s = {"op": op, "case": dict(case), "turn": 0}

    def table(B, width):
        return torch.randperm(B * width, generator=g, device=dev).to(torch.int32).view(B, width)

    if op == "reserve":
        return _prepare_reserve(s, case, rng, g, dev)
    if op == "layout":
        B, page = case["B"], case["page"]
        lens = _spread(rng, B, case["lo"], case["hi"])
        start = [rng.randint(0, case["at"]) for _ in range(B)]
        width = (case["at"] + case["hi"]) // page + 1
        s.update(count=_i32(lens, dev), start=_i32(start, dev), page_table=table(B, width),
                 N=sum(lens) + case["pad"])
        return s
    heads, dim, t = case["heads"], case["dim"], TYPES[case["type"]]
    if op == "slots":
        B, page = case["B"], case["page"]
        lens = _spread(rng, B, case["lo"], case["hi"])
        start = [rng.randint(0, case["at"]) for _ in range(B)]
        width = (case["at"] + case["hi"]) // page + 1
        tab = table(B, width)
        s.update(_cache(g, B * width, heads, dim, page, dev))
        _ragged(s, lens, start, dev)
        s["start"] = _i32(start, dev)
        s["page_table"] = tab
        s["slots"] = tab.long()[s["request"], s["position"] // page] * page + s["position"] % page
        n = sum(lens)
        s["new_k"] = _kv(g, (n, heads, dim), dev).to(t)
        s["new_v"] = _kv(g, (n, heads, dim), dev).to(t)
        return s
    rows = heads * case["group"]
    if op == "prompt":
        _ragged(s, _spread(rng, case["B"], case["lo"], case["hi"]), [0] * case["B"], dev)
        n = s["first"][-1]
        # one projection's output, used as it lies
        x = torch.randn((n, rows + 2 * heads, dim), generator=g, device=dev)
        x[:, rows:] *= torch.exp(0.5 * torch.randn(dim, generator=g, device=dev))
        s["q"], s["k"], s["v"] = x.to(t).split((rows, heads, heads), 1)
        return s
    page = case["page"]
    lens = _spread(rng, case["chunks"], max(1, case["T"] - case["T"] // 8), case["T"])
    lens += _spread(rng, case["drafts"], max(1, case["rows"] - 2), case["rows"])
    seq = [max(n, rng.randint(case["lo"], max(case["lo"], case["hi"]))) for n in lens]
    width = max(case["lo"], case["hi"], *seq) // page + 1
    s["page_table"] = table(len(lens), width)
    s.update(_cache(g, len(lens) * width, heads, dim, page, dev))
    _ragged(s, lens, [a - n for a, n in zip(seq, lens)], dev)
    s["seq"], s["seq_lens"] = seq, _i32(seq, dev)
    s["q"] = torch.randn((sum(lens), rows, dim), generator=g, device=dev).to(t)
    return s


def _prepare_reserve(s, case, rng, g, dev):
    """Two sets of lengths in turn: requests that grow by `grow` tokens and back, and a share
    `swap` of the slots that is empty in the one or in the other."""
    B, page = case["B"], case["page"]
    lens = _spread(rng, B, case["lo"], case["hi"])
    gone = [rng.random() for _ in range(B)]
    a = [0 if x < case["swap"] else n for n, x in zip(lens, gone)]
    b = [0 if x > 1 - case["swap"] else n + case["grow"] for n, x in zip(lens, gone)]
    width = -(-(case["hi"] + case["grow"]) // page)
    # `spare` times what a mean set takes; requests that do not fit at the start are empty there
    pool = int(B * ((case["lo"] + case["hi"]) / 2 / page + 1) * (1 - case["swap"]) * case["spare"])
    pool = max(pool, width)
    held, left = [], pool
    for n in a:
        held.append(-(-n // page) if -(-n // page) <= left else 0)
        left -= held[-1]
    taken = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    first = _i32(_running(held)[:-1], dev).long()
    j = torch.arange(width, device=dev)
    at = (first[:, None] + j).clamp(max=pool - 1)
    h = _i32(held, dev)
    s["page_table"] = torch.where(j < h[:, None], taken[at], torch.full_like(taken[at], -1))
    s["held"] = h
    # the pages that nobody holds, at the list's start
    s["free"] = torch.roll(taken, -sum(held))
    s["num_free"] = _i32([pool - sum(held)], dev)
    s["tokens"] = (_i32(b, dev), _i32(a, dev))
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"reserve": _reserve, "layout": _layout, "slots": _slots, "prompt": _prompt,
            "chunk": _chunk}[s["op"]](s)


def _own(s):
    import suffix_match_drafter_amd as sfx

    op, case = s["op"], s["case"]
    if op == "reserve":
        if "pool" not in s:  # the handle over the pool's buffers
            s["pool"] = sfx.PagePool(s["free"].shape[0], case["page"],
                                     buffers=(s["free"], s["num_free"]))
        missing = s["pool"].reserve(s["page_table"], s["held"], _turn(s))
        return _pool_out(s, missing)
    if op == "layout":
        if "pool" not in s:
            s["pool"] = sfx.PagePool(s["page_table"].numel(), case["page"])
        x = s["pool"].layout(s["page_table"], s["start"], s["count"], s["N"])
        return {"offsets": x.offsets, "seq_lens": x.seq_lens, "request": x.request,
                "position": x.position, "slots": x.slots}
    if op == "prompt":
        return sfx.attend_prompt(s["q"], s["k"], s["v"], s["offsets"], window=case["window"],
                                 sinks=case["sinks"])
    if "cache" not in s:  # the handle over the cache's buffers
        s["cache"] = sfx.KVCache(s["k"].shape[0], case["page"], case["heads"], case["dim"],
                                 buffers=(s["k"], s["v"], s["k_scale"], s["v_scale"]))
    if op == "slots":
        s["cache"].write_slots(s["new_k"], s["new_v"], s["slots"])
        return _cache_out(s)
    return s["cache"].attend_packed(s["q"], s["page_table"], s["seq_lens"], s["offsets"],
                                    max_q=max(s["lens"]), window=case["window"],
                                    sinks=case["sinks"])


def _turn(s):
    """The lengths of this step: the two sets in turn."""
    x = s["tokens"][s["turn"]]
    s["turn"] ^= 1
    return x


def _pool_out(s, missing):
    return {"page_table": s["page_table"], "held": s["held"], "free": s["free"],
            "num_free": s["num_free"], "missing": missing}


def _reserve(s):
    table, held, free = s["page_table"], s["held"].long(), s["free"]
    B, width = table.shape
    pool, page = free.shape[0], s["case"]["page"]
    j = torch.arange(width, device=table.device)
    need = (_turn(s).long().clamp(min=0) + page - 1) // page
    back = (held - need).clamp(min=0)
    want = (need - held).clamp(min=0)
    fits = need <= width
    nf = s["num_free"].long()
    granted = fits & (torch.where(fits, want, 0).cumsum(0) <= nf + back.sum())
    new = torch.where(granted | (want == 0), need, held)
    # released entries in order, in a list of their own
    rel = ((j >= new[:, None]) & (j < held[:, None])).view(-1)
    nth = rel.cumsum(0) - 1
    R = nth[-1] + 1
    released = torch.empty(B * width + 1, dtype=torch.int32, device=table.device)
    released.scatter_(0, torch.where(rel, nth, B * width), table.view(-1))
    # granted entries in order: a released page, or one from the free list's end
    get = ((j >= held[:, None]) & (j < new[:, None])).view(-1)
    a = get.cumsum(0) - 1
    A = a[-1] + 1
    page_id = torch.where(a < R, released[a.clamp(0, B * width)],
                          free[(nf - 1 - (a - R)).clamp(0, pool - 1)])
    table.copy_(torch.where(get, page_id, torch.where(rel, -1, table.view(-1))).view(B, width))
    # released pages left over go behind the free list
    out = torch.cat([free, free[:1]])
    out.scatter_(0, torch.where(rel & (nth >= A), nf + nth - A, pool), released[nth.clamp(min=0)])
    free.copy_(out[:pool])
    s["held"].copy_(new)
    s["num_free"].copy_(nf + R - A)
    return _pool_out(s, torch.where(granted, 0, want).to(torch.int32))


def _layout(s):
    table, start, count, N = s["page_table"].long(), s["start"].long(), s["count"].long(), s["N"]
    B, page = count.shape[0], s["case"]["page"]
    off = torch.cat([torch.zeros_like(count[:1]), count.clamp(min=0).cumsum(0)]).clamp(max=N)
    i = torch.arange(N, device=table.device)
    req = (i[:, None] >= off[1:]).sum(1)
    live = req < B
    b = req.clamp(max=B - 1)
    pos = start[b] + i - off[b]
    at = pos // page
    slot = table[b, at.clamp(max=table.shape[1] - 1)] * page + pos % page
    none = torch.full_like(pos, -1)
    return {"offsets": off.to(torch.int32), "seq_lens": (start + off[1:] - off[:-1]).to(torch.int32),
            "request": torch.where(live, req, none).to(torch.int32),
            "position": torch.where(live, pos, none).to(torch.int32),
            "slots": torch.where(live & (at < table.shape[1]), slot, none)}


def _cache_out(s):
    return {"k": s["k"].view(torch.float8_e4m3fn), "v": s["v"].view(torch.float8_e4m3fn),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _slots(s):
    """Blocks of 32 tokens: the new tokens' exponents, the old tokens of a request's first block
    carried to its new scale."""
    case, slot = s["case"], s["slots"]
    heads, dim, page = case["heads"], case["dim"], case["page"]
    n, dev, start = slot.shape[0], slot.device, s["start"].long()
    B = start.shape[0]
    head = torch.arange(heads, device=dev)
    block = slot // 32
    first = torch.cat([torch.ones_like(block[:1], dtype=torch.bool), block[1:] != block[:-1]])
    run = first.long().cumsum(0) - 1                                    # [n]
    # the 32 tokens around each request's first position, as they are
    base = (start // 32 * 32)[:, None] + torch.arange(32, device=dev)   # [B, 32]
    pg = torch.gather(s["page_table"].long(), 1, base // page)
    old_slot = (pg * page + base % page).view(-1)
    old = (base < start[:, None]).view(-1)
    lead = s["request"]                                                 # a row's request
    cont = (s["position"] // 32 == (start // 32)[lead]) & ((start % 32) != 0)[lead]
    places, old_places = _place(slot, heads, dim, page), _place(old_slot, heads, dim, page)

    def one(name, x, at, old_at):
        x, scale = x.float(), s[name + "_scale"]
        sc = ((slot // page)[:, None], head, (slot % page // 32)[:, None])
        amax = torch.zeros((n, heads), device=dev).scatter_reduce_(
            0, run[:, None].expand(n, heads), x.abs().amax(2), "amax")
        e = _exponent(amax)[run]                                        # [n, heads]
        s_old = scale[sc]
        s_new = torch.where(cont[:, None], torch.maximum(_pow2(e), s_old), _pow2(e))
        c_old = s[name][old_at]
        osc = ((old_slot // page)[:, None], head, (old_slot % page // 32)[:, None])
        before = scale[osc]
        scale[sc] = s_new
        moved = c_old.view(torch.float8_e4m3fn).float() * (before / scale[osc])[:, :, None]
        moved = torch.where(old[:, None, None], _code(moved).view(torch.uint8), c_old)
        s[name][old_at] = moved
        s[name][at] = _code(x / s_new[:, :, None]).view(torch.uint8)

    one("k", s["new_k"], places[0], old_places[0])
    one("v", s["new_v"], places[1], old_places[1])
    return _cache_out(s)


def _tokens(s, a, b):
    """All tokens of the pages of requests [a, b) in float32: [b - a, heads, tokens, dim] twice."""
    pt = s["page_table"][a:b].long()

    def one(name, unpack):
        x = unpack(s[name][pt])                                         # B n h page d
        x = x.contiguous().view(torch.float8_e4m3fn).float()
        B, n, h, page, d = x.shape
        x = x.view(B, n, h, page // 32, 32, d) * s[name + "_scale"][pt][..., None, None]
        return x.view(B, n, h, page, d).transpose(1, 2).reshape(B, h, n * page, d)

    return one("k", _unpack_k), one("v", _unpack_v)


def _weighted(case, q, k, v, pos):
    """q [B, T, heads * group, dim] at positions pos [B, T] (-1: no row) over k, v [B, heads, S,
    dim], in float32."""
    B, T, _, d = q.shape
    h, G, S = case["heads"], case["group"], k.shape[2]
    j = torch.arange(S, device=k.device)
    see = j <= pos[:, :, None]
    if case["window"]:
        see &= (j > pos[:, :, None] - case["window"]) | (j < case["sinks"])
    q = q.float().view(B, T, h, G, d).permute(0, 2, 1, 3, 4).reshape(B * h, T * G, d)
    x = torch.bmm(q, k.reshape(B * h, S, d).transpose(1, 2)).view(B, h, T, G, S)
    x.div_(math.sqrt(d)).masked_fill_(~see[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    z = x.sum(-1, keepdim=True)
    o = torch.bmm(x.view(B * h, T * G, S), v.reshape(B * h, S, d)).view(B, h, T, G, d)
    o = torch.where(z > 0, o / z, torch.zeros((), device=o.device))
    return o.permute(0, 2, 1, 3, 4).reshape(B, T, h * G, d)


def _padded(s, x, a, b, most):
    """Rows of requests [a, b) as [b - a, most, ...]; rows past a request's own are others'."""
    at = s["offsets"][a:b].long()[:, None] + torch.arange(most, device=x.device)
    return x[at.clamp(max=x.shape[0] - 1)]


def _prompt(s):
    B, most, dev = s["case"]["B"], max(s["lens"]), s["q"].device
    t = torch.arange(most, device=dev)
    n = (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    pos = torch.where(t < n, t, torch.full_like(t, -1))
    k, v = (_padded(s, s[x], 0, B, most).float().transpose(1, 2) for x in "kv")
    o = _weighted(s["case"], _padded(s, s["q"], 0, B, most), k, v, pos)
    return o[s["request"], s["row"]].to(s["q"].dtype)


def _chunk(s):
    """The chunks and the drafts, each kind padded to its longest."""
    nc, B = s["case"]["chunks"], len(s["lens"])

    def some(a, b):
        most = max(s["lens"][a:b], default=0)
        if a == b:
            return s["q"][:0]
        t = torch.arange(most, device=s["q"].device)
        n = (s["offsets"][1:] - s["offsets"][:-1])[a:b, None]
        pos = torch.where(t < n, s["seq_lens"][a:b, None] - n + t, -1)
        o = _weighted(s["case"], _padded(s, s["q"], a, b, most), *_tokens(s, a, b), pos)
        at = slice(s["first"][a], s["first"][b])
        return o[s["request"][at] - a, s["row"][at]].to(s["q"].dtype)

    return torch.cat([some(0, nc), some(nc, B)])


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(lo, hi, before_lo, before_hi, window, sinks):
    """Mean number of (row, visible token) pairs of a request of lo to hi rows behind before_lo to
    before_hi tokens."""
    n = (lo + hi) / 2
    before = (before_lo + before_hi) / 2
    square = (lo * lo + lo * hi + hi * hi) / 3
    full = n * before + (square + n) / 2
    if not window:
        return full
    return min(full, n * (window + sinks))


def work(case):
    op = case["op"]
    if op == "reserve":
        # lengths and counts read, counts and shortages written; pages that change hands
        per = case["swap"] * (case["lo"] + case["hi"]) / 2 + case["grow"] * (1 - case["swap"])
        return {"bytes": case["B"] * (16 + 12 * per / case["page"]),
                "flops": 4.0 * case["B"]}
    if op == "layout":
        n = case["B"] * (case["lo"] + case["hi"]) / 2
        return {"bytes": case["B"] * 16 + 4 * n / case["page"] + (n + case["pad"]) * 16,
                "flops": 4.0 * n}
    tok = 2 * case["heads"] * case["dim"]
    if op == "slots":
        n = case["B"] * (case["lo"] + case["hi"]) / 2
        return {"bytes": n * (tok * (1 + SIZE[case["type"]]) + 8), "flops": 2 * n * tok}
    d, rows, es = case["dim"], case["heads"] * case["group"], SIZE[case["type"]]
    win, sinks = case["window"], case["sinks"]
    if op == "prompt":
        n = case["B"] * (case["lo"] + case["hi"]) / 2
        pairs = case["B"] * _pairs(case["lo"], case["hi"], 0, 0, win, sinks)
        return {"bytes": n * (2 * rows * d + tok) * es, "flops": 4 * pairs * rows * d}
    t_lo, t_hi = max(1, case["T"] - case["T"] // 8), case["T"]
    r_lo, r_hi = max(1, case["rows"] - 2), case["rows"]
    lo, hi = case["lo"], max(case["lo"], case["hi"])
    t, r = (t_lo + t_hi) / 2, (r_lo + r_hi) / 2
    pairs = case["chunks"] * _pairs(t_lo, t_hi, max(0, lo - t), max(0, hi - t), win, sinks) + \
        case["drafts"] * _pairs(r_lo, r_hi, max(0, lo - r), max(0, hi - r), win, sinks)
    seen = (lo + hi) / 2
    read = case["chunks"] * (min(seen, win + t + sinks) if win else seen) + \
        case["drafts"] * (min(seen, win + r + sinks) if win else seen)
    n = case["chunks"] * t + case["drafts"] * r
    return {"bytes": read * tok + n * 2 * rows * d * es, "flops": 4 * pairs * rows * d}


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
    p, o = s["page_table"][b].long()[pos // page], pos % page
    D = torch.arange(dim, device=pos.device)[None, None, :]
    h = torch.arange(heads, device=pos.device)
    P, O, H = p[:, None, None], o[:, None, None], h[None, :, None]
    w = O % 32
    ik = (P, H, D // 64, O, D % 64)
    iv = (P, H, O // 32, D // 32, D % 32 // 2, w % 16 // 4, D % 2, w // 16, w % 4)
    sc = (p[:, None], h[None], (o // 32)[:, None])
    return {"k": (ik, tab[s["k"][ik].long()], s["k_scale"][sc].double()),
            "v": (iv, tab[s["v"][iv].long()], s["v_scale"][sc].double()), "scale_at": sc}


def _exact_attention(case, q, k, v, before):
    """One request: q [n, heads * group, dim], k and v [before + n, heads, dim] in 64 bits."""
    n, L, d, G = q.shape[0], k.shape[0], case["dim"], case["group"]
    out = torch.zeros((n, case["heads"] * G, d), dtype=torch.float64, device=q.device)
    at = torch.arange(L, device=q.device)
    step = max(1, (1 << 28) // max(1, G * L))
    for h in range(case["heads"]):
        kh, vh = k[:, h].contiguous(), v[:, h].contiguous()
        for r in range(0, n, step):
            part = q[r:r + step, h * G:(h + 1) * G].double()
            m = part.shape[0]
            x = (part.reshape(-1, d) @ kh.t()).view(m, G, L) / math.sqrt(d)
            pos = before + r + torch.arange(m, device=q.device)[:, None]
            see = at <= pos
            if case["window"]:
                see = see & ((at > pos - case["window"]) | (at < case["sinks"]))
            x = torch.where(see[:, None], x, torch.full_like(x, -math.inf))
            p = torch.softmax(x, -1).nan_to_num(0.0)
            out[r:r + step, h * G:(h + 1) * G] = (p.reshape(-1, L) @ vh).view(m, G, d)
    return out


def exact(case, seed):
    op = case["op"]
    if op in ("reserve", "layout"):
        return None  # whole numbers
    s = prepare(case, seed)
    dev = s["k"].device
    if op == "slots":
        return _exact_slots(s, case, dev)
    parts = []
    for b, n in enumerate(s["lens"]):
        rows = slice(s["first"][b], s["first"][b] + n)
        if op == "prompt":
            k, v, before = s["k"][rows].double(), s["v"][rows].double(), 0
        else:
            got = _at(s, b, torch.arange(s["seq"][b], device=dev))
            k, v = (got[x][1] * got[x][2][:, :, None] for x in "kv")
            before = s["seq"][b] - n
        parts.append(_exact_attention(case, s["q"][rows], k, v, before))
    return torch.cat(parts)


def _exact_slots(s, case, dev):
    tab = _value_of_byte(dev)
    out = {"k": tab[s["k"].long()], "v": tab[s["v"].long()],
           "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double()}
    for b, n in enumerate(s["lens"]):
        a = int(s["start"][b])
        first = a // 32 * 32
        got = _at(s, b, torch.arange(first, a + n, device=dev))
        for name in "kv":
            idx, val, sc = got[name]
            val = val * sc[:, :, None]
            fresh = s["new_" + name][s["first"][b]:s["first"][b] + n].double()
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
