"""Plain numpy models, in 64 bits, of the block-quantised key/value cache and its attention."""
import numpy as np

BLOCK = {"q8_0": 34, "q4_0": 18}


def quantize(x, kind):
    """(q, d16) of rows x [..., D] in f32 (bf16 values exactly), as mmq.h defines them: whole numbers
    [..., D/32, 32] and f16 scales [..., D/32]. Every step is f32, as there."""
    x = np.asarray(x, np.float32)
    x = x.reshape(*x.shape[:-1], -1, 32)
    if kind == "q8_0":
        d = np.abs(x).max(-1) / np.float32(127)
    else:
        d = np.take_along_axis(x, np.abs(x).argmax(-1)[..., None], -1)[..., 0] / np.float32(-8)
    big = np.float32(np.finfo(np.float32).max)
    with np.errstate(divide="ignore", over="ignore"):
        di = np.where(d == 0, np.float32(0), np.clip(np.float32(1) / d, -big, big)).astype(np.float32)
        q = np.rint(x * di[..., None])
        lo, hi = (-128, 127) if kind == "q8_0" else (-8, 7)
        return np.clip(q, lo, hi).astype(np.int64), d.astype(np.float16)


def value_of(q, d16):
    """The values that whole numbers and scales stand for, [..., D] in 64 bits."""
    x = q.astype(np.float64) * d16.astype(np.float64)[..., None]
    return x.reshape(*x.shape[:-2], -1)


def _nibble(i):
    return (i % 8) // 2 + 4 * (i % 2)


def store(record, t, q, d16, kind, side):
    """Token t's whole numbers [D/32, 32] and scales [D/32] into a record (uint8), by mmq.h's addresses."""
    NB = q.shape[0]
    D = 32 * NB
    r, h, a, s = t % 16, t // 16, (t % 16) // 4, 4 * (t // 16) + t % 4
    n = D * (32 if kind == "q8_0" else 16)
    for b in range(NB):
        for i in range(32):
            if kind == "q8_0":
                if side == "k":
                    at = ((h * (D // 64) + b // 2) * 64 + (i // 8) * 16 + r) * 16 + (b % 2) * 8 + i % 8
                else:
                    at = (b * 64 + a * 16 + i % 16) * 16 + (i // 16) * 8 + s
                record[at] = q[b, i] + 128
                continue
            if side == "k":
                at = (((b // 2) * 64 + (i // 8) * 16 + r) * 2 + h) * 8 + (b % 2) * 4 + _nibble(i) // 2
                shift = 4 * (_nibble(i) % 2)
            else:
                at = ((b // 2) * 64 + a * 16 + i % 16) * 16 + (b % 2) * 8 + 4 * (t // 16) + (t % 4) // 2 + 2 * (t % 2)
                shift = 0 if i < 16 else 4
            record[at] = (int(record[at]) & ~(15 << shift) & 255) | (int(q[b, i]) + 8) << shift
        at = n + 2 * ((a * NB + b) * 8 + s)
        record[at:at + 2] = np.frombuffer(np.float16(d16[b]).tobytes(), np.uint8)


def write(cache, x, slots, kind, side):
    """Rows x [rows, heads, D] into a cache [pages, heads, page/32, record] (uint8, changed in place): store() of
    every row whose slot is in the cache, all at once."""
    pages, heads, tiles, rec = cache.shape
    D = x.shape[2]
    slots = np.asarray(slots, np.int64)
    keep = np.nonzero((slots >= 0) & (slots < pages * tiles * 32))[0]
    if keep.size == 0:
        return
    q, d = quantize(np.asarray(x)[keep], kind)
    slot, head = slots[keep][:, None, None, None], np.arange(heads)[None, :, None, None]
    base = ((slot // (32 * tiles) * heads + head) * tiles + slot // 32 % tiles) * rec
    t = slot % 32
    b, i = np.arange(D // 32)[None, None, :, None], np.arange(32)[None, None, None, :]
    r, h, a, s = t % 16, t // 16, (t % 16) // 4, 4 * (t // 16) + t % 4
    n = D * (32 if kind == "q8_0" else 16)
    flat = cache.reshape(-1)
    if kind == "q8_0":
        if side == "k":
            at = ((h * (D // 64) + b // 2) * 64 + (i // 8) * 16 + r) * 16 + (b % 2) * 8 + i % 8
        else:
            at = (b * 64 + a * 16 + i % 16) * 16 + (i // 16) * 8 + s
        flat[base + at] = (q + 128).astype(np.uint8)
    else:
        if side == "k":
            at = (((b // 2) * 64 + (i // 8) * 16 + r) * 2 + h) * 8 + (b % 2) * 4 + _nibble(i) // 2
            shift = 4 * (_nibble(i) % 2)
        else:
            at = ((b // 2) * 64 + a * 16 + i % 16) * 16 + (b % 2) * 8 + 4 * (t // 16) + (t % 4) // 2 + 2 * (t % 2)
            shift = 4 * (i // 16)
        at, shift = np.broadcast_to(base + at, q.shape), np.broadcast_to(shift, q.shape)
        for half in (0, 4):                             # the lower nibbles, then the upper
            of = shift == half
            flat[at[of]] = (flat[at[of]] & (240 if half == 0 else 15)) | ((q[of] + 8) << half).astype(np.uint8)
    at = (base + n)[..., 0] + 2 * ((a[..., 0] * (D // 32) + b[..., 0]) * 8 + s[..., 0])
    bits = np.ascontiguousarray(d).view(np.uint16)
    flat[at], flat[at + 1] = (bits & 255).astype(np.uint8), (bits >> 8).astype(np.uint8)


def load(cache, kind, side):
    """Every slot's values, [pages * page, heads, D] in 64 bits, by the same addresses."""
    pages, heads, tiles, rec = cache.shape
    D = rec // BLOCK[kind]
    t, b, i = np.meshgrid(np.arange(32), np.arange(D // 32), np.arange(32), indexing="ij")
    r, h, a, s = t % 16, t // 16, (t % 16) // 4, 4 * (t // 16) + t % 4
    n = D * (32 if kind == "q8_0" else 16)
    if kind == "q8_0":
        if side == "k":
            at = ((h * (D // 64) + b // 2) * 64 + (i // 8) * 16 + r) * 16 + (b % 2) * 8 + i % 8
        else:
            at = (b * 64 + a * 16 + i % 16) * 16 + (i // 16) * 8 + s
        q = cache[..., at].astype(np.float64) - 128
    else:
        if side == "k":
            at = (((b // 2) * 64 + (i // 8) * 16 + r) * 2 + h) * 8 + (b % 2) * 4 + _nibble(i) // 2
            shift = 4 * (_nibble(i) % 2)
        else:
            at = ((b // 2) * 64 + a * 16 + i % 16) * 16 + (b % 2) * 8 + 4 * (t // 16) + (t % 4) // 2 + 2 * (t % 2)
            shift = 4 * (i // 16)
        q = (cache[..., at] >> shift & 15).astype(np.float64) - 8
    d = np.ascontiguousarray(cache[..., n:]).view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):
        x = q * d[..., (a * (D // 32) + b) * 8 + s]                 # [pages, heads, tiles, 32, D/32, 32]
    return x.transpose(0, 2, 3, 1, 4, 5).reshape(pages * tiles * 32, heads, D)


def attn(q, k, v, table, lens, starts, page, pages, max_q, mask, scale, backwards=False):
    """(out, bound) of attention: out [rows, heads_q, D] in 64 bits, NaN for rows that are not computed,
    from q [rows, heads_q, D] and the slots' values k, v [slots, heads, D]; and the sums of magnitudes
    that the bounds of errors are made of: (sum p |v|, max |score|'s terms sum |q k| scale). backwards: of two
    sequences with a row in common the first has it, not the last."""
    rows, heads_q, D = q.shape
    G = heads_q // k.shape[1]
    out = np.full(q.shape, np.nan)
    mag, terms = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in sorted(range(len(lens)), reverse=backwards):
        first, end = int(starts[b]), int(starts[b + 1])
        if not 0 <= first <= end <= rows:
            continue
        n, length = end - first, max(int(lens[b]), 0)
        for i in range(min(n, max_q)):
            slots = []
            for pos in range(min(length, len(table[b]) * page)):
                ahead = pos - (length - n)
                if ahead >= 0 and not (ahead <= i if mask is None else ahead < 64 and int(mask[first + i]) >> ahead & 1):
                    continue
                p = int(table[b][pos // page])
                if 0 <= p < pages:
                    slots.append(p * page + pos % page)
            for h in range(heads_q):
                if not slots:
                    out[first + i, h] = 0
                    continue
                kk, vv = k[slots, h // G], v[slots, h // G]
                s = scale * (kk @ q[first + i, h])
                p = np.exp(s - s.max())
                out[first + i, h] = p @ vv / p.sum()
                mag[first + i, h] = p @ np.abs(vv) / p.sum()
                terms[first + i, h] = scale * (np.abs(kk) @ np.abs(q[first + i, h])).max()
    return out, mag, terms
