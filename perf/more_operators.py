"""Cases and plain forms of the block-quantised key/value cache and the attention that reads it.

Three operators, between the projection that makes queries, keys and values and the one that takes
the heads' results:

* write - a step's keys and values quantised to q8_0 or q4_0 blocks as they go into the paged cache,
  and the same rows read back
      q8_0: d = max|x| / 127, q = rint(x / d);  q4_0: d = peak / -8, q = rint(x / d) + 8 in 0..15
* read - rows of the cache as f32 or bf16 values, by their slots
* attn - attention over the cache: one new token a sequence, a chain of them, or a tree of drafted
  ones in which a token sees the sequence before the tree and its own ancestors
      out = sum_t softmax_t(scale <q, k_t>) v_t   over the tokens t that the row sees

The state holds what a program has before the call: the cache in its documented layout (slots that
were never written hold 0xFF bytes), its table of pages, the rows of a projection's output.
"""
import math

import torch

own = False

TILE = 32           # tokens of a record, and values of a block
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"q8_0": 34, "q4_0": 18}        # a block's: its values and its f16 scale
FLT_MAX = 3.4028234663852886e38


# --------------------------------------------------------------------------------- the cases

def listed():
    def rows(op, name, **k):
        return dict(dict(name=name, op=op, heads=8, D=128, page=64, k="q8_0", v="q8_0", dtype="f32", away=0.0), **k)

    def attn(name, **k):
        return dict(dict(name=name, op="attn", heads=8, G=4, D=128, page=64, k="q8_0", v="q8_0", dtype="f32",
                         B=1, new_lo=1, new_hi=1, tree=False), **k)
    return [
        # one token of one request: latency
        rows("write", "write_1", rows=1),
        # a decode batch of 200 requests after a W8A8 projection, values in four bits
        rows("write", "write_200", rows=200, heads=5, D=64, page=32, v="q4_0", dtype="bf16"),
        # a long prompt's keys and values
        rows("write", "write_2048", rows=2048),
        # the accepted tokens of many trees: one row of four is kept, odd sizes
        rows("write", "write_1517", rows=1517, heads=3, D=192, page=128, k="q4_0", v="q4_0", dtype="bf16", away=0.75),
        # a whole context read back for a prompt's own products
        rows("read", "read_32768", rows=32768, dtype="bf16"),
        # a short, ragged one from the middle of a page
        rows("read", "read_1003", rows=1003, heads=4, D=256, page=32, k="q4_0", v="q4_0"),
        # one token of one request: latency
        attn("attn_1", len_lo=777, len_hi=777),
        # a decode batch of requests of all lengths
        attn("attn_64", B=64, len_lo=128, len_hi=8192),
        # one long context, values in four bits
        attn("attn_long", len_lo=131072, len_hi=131072, v="q4_0", dtype="bf16", page=256),
        # trees of up to 64 drafted tokens
        attn("attn_tree_8", B=8, new_lo=48, new_hi=64, tree=True, len_lo=1024, len_hi=8192, dtype="bf16"),
        # small trees, seven query heads for each of the cache, odd lengths
        attn("attn_tree_3", B=3, new_lo=5, new_hi=13, tree=True, len_lo=61, len_hi=2999, D=64, heads=2, G=7,
             page=32, k="q4_0", v="q4_0"),
        # a piece of a long prompt
        attn("attn_chunk", new_lo=512, new_hi=512, len_lo=4096, len_hi=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attn", "attn", "attn"])
    c = dict(op=op, heads=rng.choice([1, 2, 3, 4, 5, 8, 8, 16]), D=rng.choice([64, 128, 128, 192, 256]),
             page=rng.choice([32, 64, 128, 256]), k=rng.choice(["q8_0", "q4_0"]), v=rng.choice(["q8_0", "q4_0"]),
             dtype=rng.choice(["f32", "bf16"]))
    width = c["heads"] * c["D"]
    if op == "write":
        c["rows"] = min(_log(rng, 1, 2048), 2048 * 1024 // width)
        c["away"] = rng.choice([0.0, 0.0, 0.75])
    elif op == "read":
        c["rows"] = min(_log(rng, 1, 32768), 32768 * 1024 // width)
        c["away"] = rng.choice([0.0, 0.0, 0.25])
    else:
        c["G"], c["B"] = rng.choice([1, 2, 4, 4, 5, 7, 8]), _log(rng, 1, 64)
        kind = rng.choice(["token", "tree", "chain"])
        c["tree"] = kind == "tree"
        new = 1 if kind == "token" else _log(rng, 2, 64) if kind == "tree" else _log(rng, 2, 512)
        # no more values in the cache than the long case's, padded, and no more products than the chunk's
        hi = min(_log(rng, 16, 131072), 131072 * 1024 // (c["B"] * width))
        hi = max(1, min(hi, 512 * 4096 * 4096 // (c["B"] * new * c["G"] * width)))
        new = max(1, min(new, hi))
        c.update(new_lo=max(1, new // 2), new_hi=new, len_lo=max(1, new, hi // rng.choice([1, 4, 16])), len_hi=hi)
    return c


def _lens(c):
    """The sequences' lengths, the new tokens among them: from len_lo to len_hi by equal factors, shuffled."""
    B = c["B"]
    step = math.log(c["len_hi"] / c["len_lo"]) / max(1, B - 1)
    lens = [int(round(c["len_lo"] * math.exp(step * i))) if B > 1 else c["len_hi"] for i in range(B)]
    return [lens[(i * 29) % B] if B % 29 else lens[i] for i in range(B)]


def _news(c):
    """The sequences' numbers of new tokens."""
    return [c["new_lo"] + (i * 5) % (c["new_hi"] - c["new_lo"] + 1) for i in range(c["B"])]


# ------------------------------------------------------------------------------- the inputs

def _normal(g, shape):
    return torch.randn(shape, generator=g, device="cuda")


def _values(g, rows, heads, D):
    """Rows of keys or values: N(0,1), every head with a few channels eight times as large."""
    big = torch.rand((heads, D), generator=g, device="cuda") < 0.02
    return _normal(g, (rows, heads, D)) * torch.where(big, 8.0, 1.0)


def _quantize(x, kind):
    """(whole numbers, f16 scales) of the blocks of 32 values of x [..., D] in f32: [..., D/32, 32] and
    [..., D/32]. Quotients in 64 bits, rounded to f32, are the correctly rounded ones."""
    x = x.unflatten(-1, (-1, TILE))
    if kind == "q8_0":
        d = (x.abs().amax(-1).double() / 127).float()
    else:
        at = x.abs().argmax(-1, keepdim=True)
        d = (x.gather(-1, at)[..., 0].double() / -8).float()
    di = torch.where(d == 0, 0.0, (1 / d.double()).clamp(-FLT_MAX, FLT_MAX).float())
    q = (x * di[..., None]).round()
    return (q.clamp(-128, 127) if kind == "q8_0" else q.clamp(-8, 7)).to(torch.int8), d.half()


def _records(q, d, kind, side):
    """Records [pages, heads, page/32, bytes] from whole numbers q + 128 (q8_0) or q + 8 (q4_0) as uint8
    [pages, page, heads, D/32, 32] and scales f16 [pages, page, heads, D/32]."""
    P, page, H, NB, _ = q.shape
    T = page // TILE
    s = d.view(P, T, 2, 4, 4, H, NB).permute(0, 5, 1, 3, 6, 2, 4).reshape(P, H, T, -1).view(torch.uint8)
    if side == "k":
        w = q.view(P, T, 2, 16, H, NB // 2, 2, 4, 8)               # page, tile, h, r, head, bp, par, g, j
        if kind == "q8_0":
            w = w.permute(0, 4, 1, 2, 5, 7, 3, 6, 8)
        else:
            w = w[..., [0, 4, 1, 5]] | (w[..., [2, 6, 3, 7]] << 4)
            w = w.permute(0, 4, 1, 5, 7, 3, 2, 6, 8)
    else:
        w = q.view(P, T, 2, 4, 4, H, NB, 2, 16)                    # page, tile, hi, g, lo, head, b, u, r
        if kind == "q8_0":
            w = w.permute(0, 5, 1, 6, 3, 8, 7, 2, 4)
        else:
            w = (w[..., 0, :] | (w[..., 1, :] << 4))[:, :, :, :, [0, 2, 1, 3]]
            w = w.unflatten(6, (NB // 2, 2)).permute(0, 5, 1, 6, 3, 8, 7, 2, 4)
    return torch.cat([w.reshape(P, H, T, -1), s], 3)


def _filled(g, kind, side, page, heads, D, pages, count):
    """A cache of `pages` pages whose page p holds count[p] tokens from its start on; 0xFF elsewhere."""
    x = _values(g, pages * page, heads, D)
    q, d = _quantize(x, kind)
    q = (q.to(torch.int16) + (128 if kind == "q8_0" else 8)).to(torch.uint8).view(pages, page, heads, D // TILE, TILE)
    d = d.view(pages, page, heads, D // TILE)
    there = (torch.arange(page, device="cuda") < count[:, None])[..., None, None]
    none = torch.full((), -1, dtype=torch.int16, device="cuda").view(torch.float16)
    q = torch.where(there[..., None], q, 255 if kind == "q8_0" else 15)
    return _records(q, torch.where(there, d, none), kind, side).contiguous()


def _tree_masks(g, news):
    """Each drafted token's ancestors and itself, as bits: random parents among the tokens before it."""
    pick = torch.rand((sum(news),), generator=g, device="cuda").tolist()
    masks, first = [], 0
    for n in news:
        seen = []
        for i in range(n):
            parent = int(pick[first + i] * (i + 1)) - 1
            seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        masks += [m - (1 << 64) if m >> 63 else m for m in seen]
        first += n
    return torch.tensor(masks, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 6007 + 29)
    H, D, page = c["heads"], c["D"], c["page"]
    s = dict(case=dict(c), op=c["op"])
    if c["op"] != "attn":
        # a sequence whose pages lie anywhere; its rows start in the middle of a page
        n, first = c["rows"], page // 2 + 3
        pages = (first + n + page - 1) // page + 2
        where = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(first, first + n, device="cuda")
        slots = (where[at // page] * page + at % page).int()
        away = torch.rand((n,), generator=g, device="cuda") < c["away"]
        away[0] = False
        s["slots"] = torch.where(away, -1, slots)
        full = torch.full((pages,), page if c["op"] == "read" else 0, device="cuda")
        for side in "kv":
            s[side + "cache"] = _filled(g, c[side], side, page, H, D, pages, full)
        if c["op"] == "write":
            # two query heads for each of the cache, then keys, then values: a projection's rows
            x = torch.cat([_normal(g, (n, 2 * H, D)), _values(g, n, H, D), _values(g, n, H, D)], 1).to(DT[c["dtype"]])
            s["k"], s["v"] = x[:, 2 * H:3 * H], x[:, 3 * H:]
        out = torch.float32 if c["op"] == "write" else DT[c["dtype"]]
        for side in "kv":
            s[side + "_back"] = torch.zeros((n, H, D), dtype=out, device="cuda")
        return s
    lens, news = _lens(c), _news(c)
    need = [(n + page - 1) // page for n in lens]
    total, width = sum(need) + 2, max(need) + 1
    perm = torch.randperm(total, generator=g, device="cuda").tolist()
    table, count, used = [], [0] * total, 0
    for n, k in zip(lens, need):
        mine = perm[used:used + k]
        used += k
        for i, p in enumerate(mine):
            count[p] = min(page, n - i * page)
        table.append(mine + [-1] * (width - k))
    count = torch.tensor(count, device="cuda")
    for side in "kv":
        s[side + "cache"] = _filled(g, c[side], side, page, H, D, total, count)
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["starts"] = torch.tensor([0] + news, device="cuda").cumsum(0).int()
    s["max_q"] = max(news)
    rows = sum(news)
    s["q"] = _normal(g, (rows, (c["G"] + 2) * H, D)).to(DT[c["dtype"]])[:, :c["G"] * H]
    s["mask"] = _tree_masks(g, news) if c["tree"] else None
    return s


# ------------------------------------------------------------------------------- plain forms

def _decode(rec, kind, side, D):
    """Values f32 [..., 32, D] of records [..., bytes]."""
    lead, NB, n = rec.shape[:-1], D // TILE, D * (TILE if kind == "q8_0" else TILE // 2)
    w, s = rec[..., :n], rec[..., n:].contiguous().view(torch.float16)
    s = s.view(-1, 4, NB, 2, 4).permute(0, 3, 1, 4, 2).reshape(-1, TILE, NB).float()        # token, block
    if kind == "q8_0":
        if side == "k":
            w = w.reshape(-1, 2, NB // 2, 4, 16, 2, 8).permute(0, 1, 4, 2, 5, 3, 6)
        else:
            w = w.reshape(-1, NB, 4, 16, 2, 2, 4).permute(0, 5, 2, 6, 1, 4, 3)
        q = w.reshape(-1, TILE, NB, TILE).float() - 128
    else:
        if side == "k":
            w = w.reshape(-1, NB // 2, 4, 16, 2, 2, 4)                                      # bp, g, r, h, par, byte
            w = torch.stack([w & 15, w >> 4], -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]]
            w = w.permute(0, 4, 3, 1, 5, 2, 6)
        else:
            w = w.reshape(-1, NB // 2, 4, 16, 2, 2, 4)[..., [0, 2, 1, 3]]                   # bp, g, r, par, hi, lo
            w = torch.stack([w & 15, w >> 4], -1).permute(0, 5, 2, 6, 1, 4, 7, 3)
        q = w.reshape(-1, TILE, NB, TILE).float() - 8
    return (q * s[..., None]).reshape(*lead, TILE, D)


def _rows(cache, slots, kind, side, D):
    """Values f32 [rows, heads, D] at the slots."""
    NB, n = D // TILE, D * (TILE if kind == "q8_0" else TILE // 2)
    slot = slots.long()
    at = (slot // (cache.shape[2] * TILE), slice(None), slot // TILE % cache.shape[2])
    t = slot % TILE
    h, r, g, lo = t // 16, t % 16, t % 16 // 4, t % 4
    w, every = cache[..., :n], slice(None)
    if side == "k" and kind == "q8_0":
        q = w.unflatten(-1, (2, NB // 2, 4, 16, 2, 8))[(*at, h, every, every, r)]       # bp, g, par, j
        q = q.transpose(3, 4).reshape(*q.shape[:2], NB, TILE).float() - 128
    elif side == "k":
        q = w.unflatten(-1, (NB // 2, 4, 16, 2, 2, 4))[(*at, every, every, r, h)]       # bp, g, par, byte
        q = torch.stack([q & 15, q >> 4], -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]]
        q = q.transpose(3, 4).reshape(*q.shape[:2], NB, TILE).float() - 8
    elif kind == "q8_0":
        q = w.unflatten(-1, (NB, 4, 16, 2, 2, 4))[(*at, every, g, every, every, h, lo)]  # b, r, u
        q = q.transpose(3, 4).reshape(*q.shape[:2], NB, TILE).float() - 128
    else:
        byte = lo // 2 + lo % 2 * 2
        q = w.unflatten(-1, (NB // 2, 4, 16, 2, 2, 4))[(*at, every, g, every, every, h, byte)]  # bp, r, par
        q = torch.stack([q & 15, q >> 4], 3)                                            # bp, u, r, par
        q = q.permute(0, 1, 2, 5, 3, 4).reshape(*q.shape[:2], NB, TILE).float() - 8
    d = cache.view(torch.float16)[..., n // 2:].unflatten(-1, (4, NB, 2, 4))[(*at, g, every, h, lo)]
    return (q * d.float()[..., None]).flatten(-2)


def _plain_read(s, dtype):
    """The slots' rows; zeros for rows without a slot."""
    c, slot, there = s["case"], s["slots"].clamp(min=0), (s["slots"] >= 0)[:, None, None]
    k = _rows(s["kcache"], slot, c["k"], "k", c["D"])
    v = _rows(s["vcache"], slot, c["v"], "v", c["D"])
    return {"k": torch.where(there, k, 0.0).to(dtype), "v": torch.where(there, v, 0.0).to(dtype)}


def _put(cache, x, slots, kind, side, D):
    """Rows x [rows, heads, D] quantised and stored into their slots."""
    keep = torch.nonzero(slots >= 0)[:, 0]
    slot, x = slots[keep].long(), x[keep].float()
    _, H, T, rec = cache.shape
    NB, n = D // TILE, D * (TILE if kind == "q8_0" else TILE // 2)
    q, d = _quantize(x, kind)
    q = q.to(torch.int16) + (128 if kind == "q8_0" else 8)
    t = (slot % TILE)[:, None, None, None]
    base = ((slot // (T * TILE) * H)[:, None] + torch.arange(H, device="cuda")) * T + (slot // TILE % T)[:, None]
    base = (base * rec)[:, :, None, None]
    b = torch.arange(NB, device="cuda")[:, None]
    i = torch.arange(TILE if kind == "q8_0" else TILE // 2, device="cuda")
    if side == "k" and kind == "q8_0":
        at = (((t // 16) * (NB // 2) + b // 2) * 64 + i // 8 * 16 + t % 16) * 16 + b % 2 * 8 + i % 8
    elif side == "k":
        q = q.unflatten(-1, (4, 8))
        q = (q[..., [0, 4, 1, 5]] | (q[..., [2, 6, 3, 7]] << 4)).flatten(-2)
        at = ((b // 2 * 64 + i // 4 * 16 + t % 16) * 2 + t // 16) * 8 + b % 2 * 4 + i % 4
    elif kind == "q8_0":
        at = (b * 64 + t % 16 // 4 * 16 + i % 16) * 16 + i // 16 * 8 + t // 16 * 4 + t % 4
    else:
        q = q[..., :16] | (q[..., 16:] << 4)
        lo = t % 4 // 2 + t % 2 * 2
        at = (b // 2 * 64 + t % 16 // 4 * 16 + i) * 16 + b % 2 * 8 + t // 16 * 4 + lo
    flat = cache.view(-1)
    flat[base + at] = q.to(torch.uint8)
    at = ((t % 16 // 4 * NB + b) * 8 + t // 16 * 4 + t % 4) * 2 + n
    flat.view(torch.float16)[(base + at)[..., 0] // 2] = d


def _plain_write(s):
    c = s["case"]
    _put(s["kcache"], s["k"], s["slots"], c["k"], "k", c["D"])
    _put(s["vcache"], s["v"], s["slots"], c["v"], "v", c["D"])
    return _plain_read(s, torch.float32)


def _plain_attn(s):
    c = s["case"]
    B, H, D, G, Q = c["B"], c["heads"], c["D"], c["G"], s["max_q"]
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    page = s["table"].long().clamp(min=0)

    def tokens(side):                                          # [B, H, width * page, D]
        x = _decode(s[side + "cache"][page], c[side], side, D)
        return x.permute(0, 2, 1, 3, 4, 5).reshape(B, H, -1, D)
    k, v = tokens("k"), tokens("v")
    row = torch.arange(Q, device="cuda")
    has = row < new[:, None]                                   # [B, Q]
    at = torch.where(has, starts[:-1, None] + row, 0)
    pos = torch.arange(k.shape[2], device="cuda")
    ahead = pos - (lens - new)[:, None]                        # [B, L]: the new token at a position
    if c["tree"]:
        bit = (s["mask"][at][:, :, None] >> ahead.clamp(0, 63)[:, None]) & 1
        sees = (ahead < 0)[:, None] | ((bit == 1) & (ahead < new[:, None])[:, None])
    else:
        sees = ahead[:, None] <= row[:, None]
    sees = sees & (pos < lens[:, None])[:, None]
    v = torch.where((pos < lens[:, None])[:, None, :, None], v, 0.0)
    q = s["q"].float()[at].view(B, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, Q * G, D)
    score = (q @ k.transpose(2, 3).contiguous()).view(B, H, Q, G, -1) * D ** -0.5
    p = torch.where(sees[:, None, :, None], score, float("-inf")).softmax(-1)
    out = (p.view(B, H, Q * G, -1) @ v).view(B, H, Q, G, D).permute(0, 2, 1, 3, 4).reshape(B, Q, H * G, D)
    return {"out": out[has].to(s["q"].dtype)}


# --------------------------------------------------------------------------- the operators

def _own(s):
    import block_quantized_int8_amd as mmq
    c = s["case"]
    if c["op"] == "attn":
        return {"out": mmq.cache_attn(s["q"], s["kcache"], s["vcache"], s["table"], s["lens"], s["starts"],
                                      s["max_q"], ktype=c["k"], vtype=c["v"], mask=s["mask"])}
    if c["op"] == "write":
        mmq.cache_write(s["k"], s["v"], s["slots"], s["kcache"], s["vcache"], ktype=c["k"], vtype=c["v"])
    k, v = mmq.cache_read(s["slots"], s["kcache"], s["vcache"], ktype=c["k"], vtype=c["v"],
                          k=s["k_back"], v=s["v_back"])
    return {"k": k, "v": v}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "attn":
        return _plain_attn(state)
    return _plain_write(state) if state["op"] == "write" else _plain_read(state, DT[state["case"]["dtype"]])


# ------------------------------------------------------------------------------ in 64 bits

def _exact_rows(cache, slots, kind, side, D):
    """Values [rows, heads, D] in 64 bits at the slots, from the layout's own byte addresses."""
    _, H, T, rec = cache.shape
    NB = D // TILE
    slot = slots.long()[:, None, None]
    d = torch.arange(D, device="cuda")
    t = slot % TILE
    b, i = d // 32, d % 32
    base = ((slot // (T * TILE) * H + torch.arange(H, device="cuda")[None, :, None]) * T + slot // TILE % T) * rec
    if side == "k":
        lane = i // 8 * 16 + t % 16
        j = i % 8
        if kind == "q8_0":
            at = ((t // 16 * (NB // 2) + b // 2) * 64 + lane) * 16 + b % 2 * 8 + j
        else:
            nib = j // 2 + j % 2 * 4
            at = ((b // 2 * 64 + lane) * 2 + t // 16) * 8 + b % 2 * 4 + nib // 2
            shift = nib % 2 * 4
    else:
        lane = t % 16 // 4 * 16 + i % 16
        if kind == "q8_0":
            at = (b * 64 + lane) * 16 + i // 16 * 8 + t // 16 * 4 + t % 4
        else:
            at = (b // 2 * 64 + lane) * 16 + b % 2 * 8 + t // 16 * 4 + t % 4 // 2 + t % 2 * 2
            shift = i // 16 * 4
    flat = cache.view(-1)
    byte = flat[base + at].long()
    q = byte - 128 if kind == "q8_0" else (byte >> shift & 15) - 8
    n = D * (TILE if kind == "q8_0" else TILE // 2)
    scale = base + n + ((t % 16 // 4 * NB + b) * 8 + t // 16 * 4 + t % 4) * 2
    return q.double() * flat.view(torch.float16)[scale // 2].double()


def _exact_written(x, kind):
    """The values that rows stand for once they are quantised: whole numbers times f16 scales."""
    x = x.float().double().unflatten(-1, (-1, TILE))
    if kind == "q8_0":
        d = x.abs().amax(-1, keepdim=True) / 127
        lo, hi = -128, 127
    else:
        d = x.gather(-1, x.abs().argmax(-1, keepdim=True)) / -8
        lo, hi = -8, 7
    d = d.float().double()
    di = torch.where(d == 0, 0.0, 1 / d).float().double()
    q = (x * di).float().double().round().clamp(lo, hi)
    return (q * d.float().half().double()).flatten(-2)


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] != "attn":
        there = (s["slots"] >= 0)[:, None, None]
        if c["op"] == "write":
            return {side: torch.where(there, _exact_written(s[side], c[side]), 0.0) for side in "kv"}
        return {side: torch.where(there, _exact_rows(s[side + "cache"], s["slots"].clamp(min=0), c[side], side, c["D"]), 0.0)
                for side in "kv"}
    D, G, page, out = c["D"], c["G"], c["page"], []
    for b, (n, new) in enumerate(zip(_lens(c), _news(c))):
        pos = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[pos // page] * page + pos % page
        k = _exact_rows(s["kcache"], slots, c["k"], "k", D)
        v = _exact_rows(s["vcache"], slots, c["v"], "v", D)
        first = int(s["starts"][b])
        q = s["q"][first:first + new].double()
        i = torch.arange(new, device="cuda")
        sees = torch.ones((new, n), dtype=torch.bool, device="cuda")
        if c["tree"]:
            sees[:, n - new:] = (s["mask"][first:first + new, None] >> i & 1).bool()
        else:
            sees[:, n - new:] = i[None] <= i[:, None]
        mine = torch.empty((new, c["heads"] * G, D), dtype=torch.float64, device="cuda")
        for h in range(c["heads"] * G):
            score = q[:, h] @ k[:, h // G].T.contiguous() / math.sqrt(D)
            mine[:, h] = torch.where(sees, score, -math.inf).softmax(1) @ v[:, h // G]
        out.append(mine)
    return {"out": torch.cat(out)}


# ------------------------------------------------------------------------------------ work

def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2
    width = c["heads"] * c["D"]
    cache = width // TILE * (BYTES[c["k"]] + BYTES[c["v"]])          # bytes of a token
    if c["op"] != "attn":
        here = c["rows"] * (1 - c["away"])
        if c["op"] == "write":                                       # in, into the cache, out of it again
            return {"bytes": here * (2 * width * size + 2 * cache + 2 * width * 4) + 8 * c["rows"], "flops": 0}
        return {"bytes": here * (cache + 2 * width * size) + 4 * c["rows"], "flops": 0}
    lens, news = _lens(c), _news(c)
    pairs = sum(new * (n - new) + (new * (new + 1) // 2) for n, new in zip(lens, news))
    table = sum((n + c["page"] - 1) // c["page"] for n in lens)
    return {"bytes": sum(lens) * cache + 2 * sum(news) * c["G"] * width * size + 4 * (table + 2 * c["B"] + 1),
            "flops": 4 * pairs * c["G"] * width}
