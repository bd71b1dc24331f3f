"""The key/value cache on the GPU, through the public binding: what is written byte for byte against
the model of the layout, what is read back bit for bit, and attention against 64-bit sums.

Tolerances of attention, from the number formats (u = 2^-24, half a step of f32). With T the largest
sum of magnitudes of a score's terms, N the tokens and |o| the sum of p |v|:
  - a score is off by the split of q (2^-22 of each term, f32 rows) and by at most 2D + 24 additions
    and products of 2u each:                                             ds = (2D + 24) 2u T + 2^-22 T
  - its exponent is three roundings of numbers up to 2T + 10, the exponential 2^-22 of itself:
                                                                         e = ds + 6u (2T + 10) + 2^-22
  - numerator and denominator follow, each over N + 32 additions:        2 e + 4u (N + 32)
  - weights enter the second product to 2^-22 (two terms) or 2^-11 (one), and to 2^-25 where the
    largest weight times the largest scale is at least 2^10:             N 2^-28 max|v|
  - the result is rounded once, bf16 by at most 2^-8 of itself."""
import numpy as np
import pytest

import cachemodel
import rowmodel

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    import block_quantized_int8_amd as mmq
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mmq.lib()
    return torch, mmq


def _dtype(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _rows(r, rows, heads, D, dt):
    """Rows of very different sizes: of ordinary ones, of one value, zeros, ties of both signs."""
    x = r.standard_normal((rows, heads, D)).astype(np.float32)
    x *= np.exp2(r.integers(-6, 7, (rows, heads, D // 32, 1))).repeat(32, 3).reshape(rows, heads, D).astype(np.float32)
    if rows > 3:
        x[1] = 0.0
        x[2, :, ::2] = 1.5
        x[2, :, 1::2] = -1.5
        x[3, :, 5] = 3e4
    return x if dt == "f32" else rowmodel.bf16(x)


def _garbage(r, shape):
    """Records of slots that were never written: any bytes, among the scales NaN and infinities."""
    c = r.integers(0, 256, shape).astype(np.uint8)
    c[..., -8:] = 0xFF
    return c


ROWS = [("f32", "q8_0", "q8_0", 1, 1, 64, 32, 2), ("bf16", "q4_0", "q8_0", 5, 3, 128, 64, 3),
        ("f32", "q8_0", "q4_0", 77, 2, 192, 32, 5), ("bf16", "q4_0", "q4_0", 130, 5, 256, 128, 2),
        ("f32", "q4_0", "q4_0", 64, 4, 128, 256, 2), ("bf16", "q8_0", "q8_0", 300, 1, 64, 64, 8),
        ("f32", "q8_0", "q8_0", 259, 3, 128, 32, 12),
        # rows enough for windows of 32, and of 64
        ("f32", "q8_0", "q4_0", 1700, 8, 128, 64, 40), ("bf16", "q4_0", "q8_0", 2200, 3, 256, 32, 80),
        ("f32", "q4_0", "q8_0", 4101, 2, 192, 128, 40), ("bf16", "q8_0", "q8_0", 8200, 16, 64, 256, 40),
        ("f32", "q4_0", "q4_0", 8199, 16, 64, 64, 140)]


def _slots(r, rows, pages, page, how):
    total = pages * page
    if how == "run":                        # a sequence from the middle of a page on, its pages anywhere
        first = 3 if rows + 3 <= total else 0
        pos = first + np.arange(rows)
        slots = r.permutation(pages)[pos // page] * page + pos % page
    elif how == "tile":                     # whole records
        slots = np.arange(rows)
    else:                                   # anywhere, and nowhere
        slots = r.permutation(total)[:rows]
        slots[r.random(rows) < 0.2] = -1
        slots[r.random(rows) < 0.05] = total
        slots[r.random(rows) < 0.05] = np.iinfo(np.int32).max
        slots[r.random(rows) < 0.05] = np.iinfo(np.int32).min
    return slots.astype(np.int32)


@pytest.mark.parametrize("how", ["run", "tile", "any"])
@pytest.mark.parametrize("dt,kt,vt,rows,heads,D,page,pages", ROWS)
def test_write_and_read(env, dt, kt, vt, rows, heads, D, page, pages, how):
    torch, mmq = env
    print(f"[case] cache {dt} {kt} {vt} rows={rows} heads={heads} D={D} page={page} {how}", flush=True)
    r = np.random.default_rng([rows, D, len(how)])
    slots = _slots(r, rows, pages, page, how)
    sd = torch.from_numpy(slots).cuda()
    want, dev, rest = {}, {}, {}
    qkv = np.concatenate([_rows(r, rows, heads, D, dt) for _ in range(3)], 1)
    x = torch.from_numpy(qkv).to(_dtype(torch, dt)).cuda()               # a projection's rows: q, k, v
    for i, (side, kind) in enumerate((("k", kt), ("v", vt))):
        c = _garbage(r, mmq.cache_shape(kind, pages, page, heads, D))
        dev[side] = torch.from_numpy(c.copy()).cuda()
        cachemodel.write(c, qkv[:, (i + 1) * heads:(i + 2) * heads], slots, kind, side)
        want[side] = c
    k, v = x[:, heads:2 * heads], x[:, 2 * heads:]
    mmq.cache_write(k, v, sd, dev["k"], dev["v"], kt, vt)
    for side in "kv":
        assert np.array_equal(dev[side].cpu().numpy(), want[side]), side
    there = (slots >= 0) & (slots < pages * page)
    for out in ("f32", "bf16"):
        back = [torch.full((rows, heads * D + 3), -7.0, dtype=_dtype(torch, out), device="cuda") for _ in range(2)]
        got = mmq.cache_read(sd, dev["k"], dev["v"], kt, vt, k=back[0][:, :heads * D], v=back[1][:, :heads * D])
        assert got[0].data_ptr() == back[0].data_ptr()
        for side, kind, b in (("k", kt, back[0]), ("v", vt, back[1])):
            b = b.float().cpu().numpy()
            assert np.all(b[:, heads * D:] == -7.0) and np.all(b[~there] == -7.0)
            values = cachemodel.load(want[side], kind, side)[slots[there]].astype(np.float32)
            if out == "bf16":
                values = rowmodel.bf16(values)
            assert np.array_equal(b[there, :heads * D], values.reshape(-1, heads * D)), (side, out)


def test_read_names_a_slot_twice(env):
    torch, mmq = env
    r = np.random.default_rng(8)
    c = torch.from_numpy(r.integers(0, 100, mmq.cache_shape("q8_0", 2, 32, 2, 64)).astype(np.uint8)).cuda()
    slots = torch.tensor([5, 5, 63, 5, 0, 63], dtype=torch.int32, device="cuda")
    k, v = mmq.cache_read(slots, c, c, dtype=torch.float32)
    assert k.shape == (6, 2, 64)
    host = c.cpu().numpy()
    assert np.array_equal(k.cpu().numpy(), cachemodel.load(host, "q8_0", "k")[slots.cpu().numpy()].astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), cachemodel.load(host, "q8_0", "v")[slots.cpu().numpy()].astype(np.float32))


def test_quantisation_is_the_act_buffers(env):
    """q8_0 blocks hold what quantize_act makes of the same rows."""
    torch, mmq = env
    r = np.random.default_rng(9)
    x = _rows(r, 37, 2, 128, "f32")
    xd = torch.from_numpy(x).cuda()
    cache = [torch.zeros(mmq.cache_shape("q8_0", 2, 32, 2, 128), dtype=torch.uint8, device="cuda") for _ in range(2)]
    mmq.cache_write(xd, xd, torch.arange(37, dtype=torch.int32, device="cuda"), *cache)
    act = mmq.quantize_act(xd.view(37, 256))
    xq, xs, _ = mmq.act_to_host(act.cpu().numpy(), 37, 256)
    want = xq.astype(np.float64) * np.repeat(xs.astype(np.float64), 32, 1)
    for side, c in zip("kv", cache):
        got = cachemodel.load(c.cpu().numpy(), "q8_0", side)[:37].reshape(37, 256)
        assert np.array_equal(got, want)


# ------------------------------------------------------------------------------ attention

class Case:
    """A batch: caches with garbage in unwritten slots, tables with pages of none past the lengths."""

    def __init__(self, env, dt="f32", kt="q8_0", vt="q8_0", D=128, heads=2, G=4, page=32, lens=(70,), news=(1,), width=None,
                 tree=False, seed=1, std=1.0):
        self.torch, self.mmq = env
        torch, mmq = env
        r = self.r = np.random.default_rng([seed, D, page, sum(lens)])
        self.dt, self.kt, self.vt, self.page, self.heads, self.G, self.D = dt, kt, vt, page, heads, G, D
        need = [-(-n // page) for n in lens]
        self.width = width or max(need) + 1
        self.pages = sum(need) + 2
        perm = r.permutation(self.pages)
        table = np.full((len(lens), self.width), -1, np.int32)
        used = 0
        for b, n in enumerate(need):
            n = min(n, self.width)
            table[b, :n] = perm[used:used + n]
            used += n
        self.table, self.lens, self.news = table, np.array(lens, np.int32), list(news)
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.rows, self.max_q = int(sum(news)), max(1, max(news))
        self.host = {}
        for side, kind in (("k", kt), ("v", vt)):
            c = _garbage(r, mmq.cache_shape(kind, self.pages, page, heads, D))
            slots = np.concatenate([table[b, np.arange(min(n, self.width * page)) // page] * page +
                                    np.arange(min(n, self.width * page)) % page for b, n in enumerate(lens)])
            x = (r.standard_normal((len(slots), heads, D)) * std).astype(np.float32)
            x[:, :, 3] *= 8
            cachemodel.write(c, x, slots, kind, side)
            self.host[side] = c
        q = r.standard_normal((self.rows, heads * G + 1, D)).astype(np.float32)
        self.qh = (q if dt == "f32" else rowmodel.bf16(q))[:, :heads * G]
        self.mask = None
        if tree:
            m = []
            for n in news:
                seen = []
                for i in range(n):
                    p = int(r.integers(-1, i))
                    seen.append((seen[p] if p >= 0 else 0) | 1 << i)
                m += seen
            self.mask = np.array(m, np.uint64)
        self.scale = D ** -0.5

    def device(self):
        torch = self.torch
        pad = torch.zeros((self.rows, self.heads * self.G + 1, self.D), dtype=_dtype(torch, self.dt), device="cuda")
        pad[:, :self.heads * self.G] = torch.from_numpy(self.qh).to(pad.dtype).cuda()
        self.q = pad[:, :self.heads * self.G]
        self.kc, self.vc = (torch.from_numpy(self.host[s]).cuda() for s in "kv")
        self.td, self.ld, self.sd = (torch.from_numpy(a).cuda() for a in (self.table, self.lens, self.starts))
        self.md = None if self.mask is None else torch.from_numpy(self.mask.view(np.int64)).cuda()
        return self

    def run(self, **kw):
        return self.mmq.cache_attn(self.q, self.kc, self.vc, self.td, self.ld, self.sd, self.max_q, self.kt, self.vt,
                                   mask=self.md, scale=self.scale, **kw)

    def want(self, backwards=False):
        k, v = (cachemodel.load(self.host[s], t, s) for s, t in (("k", self.kt), ("v", self.vt)))
        with np.errstate(invalid="ignore"):
            out, mag, terms = cachemodel.attn(self.qh.astype(np.float64), k, v, self.table, self.lens, self.starts, self.page,
                                              self.pages, self.max_q, self.mask, self.scale, backwards)
        N = int(self.lens.max(initial=0))
        T = terms[:, :, None]
        ds = (2 * self.D + 24) * 2 * U24 * T + 2.0 ** -22 * T
        e = ds + 6 * U24 * (2 * T + 10) + 2.0 ** -22
        used = [p * self.page + j for b, n in enumerate(self.lens) for i, p in enumerate(self.table[b]) if 0 <= p < self.pages
                for j in range(self.page) if i * self.page + j < n]
        vmax = np.abs(v[used]).max(initial=0)
        weight = 2.0 ** -22 if self.dt == "f32" else 2.0 ** -11
        bound = mag * (2 * e + 4 * U24 * (N + 32) + weight) * 1.01 + N * 2.0 ** -28 * vmax
        bound += np.abs(out) * (U24 if self.dt == "f32" else 2.0 ** -8)
        return out, bound

    def check(self, got=None, fill=None):
        if got is None:
            buf = self.torch.full((self.rows + 2, self.heads * self.G * self.D + 5), -7.0, dtype=_dtype(self.torch, self.dt),
                                  device="cuda")
            self.run(out=buf[:self.rows, :self.heads * self.G * self.D])
            b = buf.float().cpu().numpy().astype(np.float64)
            assert np.all(b[self.rows:] == -7.0) and np.all(b[:, self.heads * self.G * self.D:] == -7.0)
            got, fill = b[:self.rows, :-5].reshape(self.qh.shape), -7.0
        want, bound = self.want()
        none = np.isnan(want)
        assert np.all(np.isfinite(got))
        if fill is not None:
            assert np.all(got[none] == fill)
        off = np.abs(got - want)[~none]
        worst = float((off / np.maximum(bound[~none], 1e-300)).max(initial=0))
        print(f"[case]   error at most {worst:.4f} of the bound", flush=True)
        assert np.all(off <= bound[~none])
        return got


ATTN = [
    dict(lens=(1,), news=(1,)),
    dict(lens=(70,), news=(1,), kt="q4_0", vt="q4_0"),
    dict(lens=(32, 33, 31, 64), news=(1, 1, 1, 1), dt="bf16"),
    dict(lens=(0, 5), news=(1, 1)),                                       # a sequence without tokens: zeros
    dict(lens=(129, 200), news=(3, 7), D=64, G=7, heads=3, vt="q4_0"),
    dict(lens=(129, 200, 90), news=(40, 1, 64), D=64, G=1, heads=2, kt="q4_0", dt="bf16"),
    dict(lens=(100, 64), news=(33, 64), tree=True, page=64),
    dict(lens=(100, 64, 65), news=(5, 64, 2), tree=True, page=128, D=192, G=2, dt="bf16", vt="q4_0"),
    dict(lens=(300,), news=(9,), tree=True, page=256, D=256, G=5, heads=1, kt="q4_0"),
    dict(lens=(3, 70), news=(5, 1)),                                       # fewer tokens than rows
    dict(lens=(3, 70), news=(5, 2), tree=True, D=64),
    dict(lens=(200, 10), news=(2, 1), width=3),                            # longer than the table
    dict(lens=(1500,), news=(2,), page=64),                                # split over chunks
    dict(lens=(900, 40, 1300, 0), news=(1, 2, 3, 1), page=64, dt="bf16", kt="q4_0", vt="q4_0", D=64),
    dict(lens=(700, 1100), news=(30, 64), tree=True, page=32, G=8, heads=1, D=64),
    dict(lens=(500,), news=(300,), D=64, heads=1, G=3, page=64),           # a piece of a prompt
    dict(lens=tuple(range(1, 300, 3)), news=(1,) * 100, D=64, heads=1, G=2),
    dict(lens=tuple((i * 37) % 97 for i in range(300)), news=tuple(i % 3 for i in range(300)), D=64, heads=1, G=1),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(f"{k}{v if not isinstance(v, tuple) or len(v) < 5 else len(v)}"
                                                              for k, v in c.items()).replace(" ", ""))
def test_attention(env, case):
    print(f"[case] attn {case if len(case['lens']) < 9 else {**case, 'lens': '..', 'news': '..'}}", flush=True)
    c = Case(env, **case).device()
    first = c.check()
    assert np.array_equal(c.run().float().cpu().numpy().reshape(first.shape).astype(np.float64)[~np.isnan(c.want()[0])],
                          first[~np.isnan(c.want()[0])])                  # the same bits again


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("std", [1e-4, 1e3])
def test_attention_of_small_and_large_values(env, dt, std):
    """Scales far from one: keys and values of 1e-4 (scales below f16's normal numbers) and of 1e3."""
    print(f"[case] attn {dt} std={std}", flush=True)
    c = Case(env, dt=dt, lens=(130, 60), news=(2, 1), D=64, std=std, seed=3)
    c.scale = 0.125 / std
    c.device().check()


def test_attention_when_value_scales_grow_and_shrink_along_the_sequence(env):
    """The products' exponent follows the largest scale so far: tiles of 1e-3, then 1, 1e3, 1."""
    c = Case(env, lens=(128 * 4,), news=(1,), D=64, heads=1, G=2, page=128, seed=4)
    x = c.r.standard_normal((512, 1, 64)).astype(np.float32) * np.repeat([1e-3, 1.0, 1e3, 1.0], 128)[:, None, None].astype(np.float32)
    slots = c.table[0, np.arange(512) // 128] * 128 + np.arange(512) % 128
    cachemodel.write(c.host["v"], x, slots, "q8_0", "v")
    c.device().check()


def test_masks_that_leave_a_row_empty_and_bits_past_the_tree(env):
    c = Case(env, lens=(6, 40), news=(6, 5), tree=True, D=64, seed=5)
    c.mask[0] = 0                                   # nothing before it, nothing of the tree: zeros
    c.mask[2] = 2 ** 64 - 1                         # bits past the sequence's tokens count nothing
    c.mask[3] = 1 << 4                              # a token that does not see itself
    c.mask[8] = 0                                   # sees what is before the tree
    got = c.device().check()
    assert np.all(got[0] == 0.0) and np.all(got[8] != 0.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_hidden_tokens_that_are_not_finite_change_nothing(env, dt):
    """A drafted token with infinite and NaN scales, seen by two rows of the tree only, which are not
    finite then; the other rows stay within the bound of what they are without it (the exponent that
    a tile's products share may differ, so not the same bits)."""
    torch, mmq = env
    c = Case(env, dt=dt, lens=(100,), news=(8,), tree=True, D=64, seed=6)
    c.mask[:] = [1 | 1 << i for i in range(8)]
    c.mask[5] |= np.uint64(1 << 3)
    c.device()
    want, bound = c.want()
    c.check()
    pos = 100 - 8 + 3
    slot = c.table[0, pos // 32] * 32 + pos % 32
    t, a = slot % 32, (slot % 16) // 4
    for cache, bits in ((c.kc, 0x7E00), (c.vc, 0x7C00)):
        rec = cache.cpu().numpy()
        for b in range(2):
            at = 64 * 32 + 2 * ((a * 2 + b) * 8 + 4 * (t // 16) + t % 4)
            rec[slot // 32, :, 0, at:at + 2] = np.frombuffer(np.uint16(bits).tobytes(), np.uint8)
        cache.copy_(torch.from_numpy(rec))
    after = c.run().float().cpu().numpy().astype(np.float64)
    others = [0, 1, 2, 4, 6, 7]
    assert np.all(np.abs(after - want)[others] <= bound[others])
    assert not np.isfinite(after[3]).any() and not np.isfinite(after[5]).any()


def test_pages_outside_the_cache_and_starts_out_of_order(env):
    """Tokens of no page are not seen; a sequence whose rows are not in the batch has none; a row that two
    sequences have holds the result of one of them."""
    c = Case(env, lens=(100, 100, 100, 100), news=(2, 3, 2, 2), D=64, seed=7)
    c.table[0, 1], c.table[0, 0] = c.pages, -5
    c.table[1, :] = np.iinfo(np.int32).max
    c.device().check()
    for starts in ([0, 2, 1, 7, 9], [-1, 2, 5, 7, 9], [0, 2, 5, 7, 10], [0, 2, 5, 9, 7]):
        c.starts = np.array(starts, np.int32)
        c.sd = c.torch.from_numpy(c.starts).cuda()
        got = c.run().cpu().numpy().astype(np.float64)
        (last, near), (first, near1) = c.want(), c.want(backwards=True)
        none = np.isnan(last)
        assert np.array_equal(none, np.isnan(first))
        assert np.all((np.abs(got - last) <= near)[~none] | (np.abs(got - first) <= near1)[~none])
    c.lens = np.array([-3, 100, np.iinfo(np.int32).max, np.iinfo(np.int32).min], np.int32)
    c.starts = np.array([0, 2, 5, 7, 9], np.int32)
    c.ld, c.sd = c.torch.from_numpy(c.lens).cuda(), c.torch.from_numpy(c.starts).cuda()
    got = c.run().cpu().numpy()
    assert np.all(got[:2] == 0.0) and np.all(got[7:] == 0.0)


def test_rows_past_max_q_are_left(env):
    c = Case(env, lens=(100, 50), news=(6, 2), D=64, seed=8)
    c.max_q = 2
    c.device().check()


def test_pages_shared_by_sequences(env):
    c = Case(env, lens=(90, 70), news=(2, 3), D=64, seed=9)
    c.table[1, :2] = c.table[0, :2]
    c.device().check()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_a_graph_replays_other_lengths(env, dt):
    """Captured once, replayed while lengths, tables and queries change in place: every replay gives
    the bits of an eager call; two graphs with workspaces of their own, and eager work between them."""
    torch, mmq = env
    cases = [Case(env, dt=dt, lens=(700, 300), news=(1, 1), D=64, page=64, seed=s, width=30).device() for s in (10, 11)]
    graphs, outs = [], []
    for c in cases:
        need = mmq.cache_attn_workspace_bytes(c.rows, c.heads * c.G, 64, c.heads, 64, 30, 2, 1)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        out = torch.empty(c.q.shape, dtype=c.q.dtype, device="cuda")
        slots = torch.tensor([c.table[b, (n - 1) // 64] * 64 + (n - 1) % 64 for b, n in enumerate(c.lens)], dtype=torch.int32,
                             device="cuda")
        new = torch.randn(2, 2, c.heads, 64, device="cuda").to(c.q.dtype)
        def step(c=c, ws=ws, out=out, slots=slots, new=new):
            mmq.cache_write(new[0], new[1], slots, c.kc, c.vc)
            c.run(out=out, workspace=ws)
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
        outs.append(out)
    for turn in range(4):
        for c, g, out in zip(cases, graphs, outs):
            c.ld[0] = 700 - 150 * turn
            c.q.copy_(torch.randn(c.q.shape, device="cuda"))
            g.replay()
        torch.cuda.synchronize()
        for c, out in zip(cases, outs):
            assert torch.equal(c.run().view(torch.uint8), out.view(torch.uint8))


def test_another_stream(env):
    torch, mmq = env
    c = Case(env, lens=(700, 300), news=(1, 1), D=64, page=64, seed=12).device()
    want = c.run().cpu()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    k, v = mmq.cache_read(slots, c.kc, c.vc, stream=s)
    s.synchronize()
    assert torch.equal(got.cpu(), want)
    k1, v1 = mmq.cache_read(slots, c.kc, c.vc)
    assert np.array_equal(k.cpu().numpy(), k1.cpu().numpy(), equal_nan=True)
    assert np.array_equal(v.cpu().numpy(), v1.cpu().numpy(), equal_nan=True)


def test_a_step_from_projection_to_projection(env):
    """Tokens quantised, projected to queries, keys and values, the cache written, attended to, and the
    result quantised and projected, against the same step in 64 bits from the quantised values."""
    torch, mmq = env
    import gen
    import oracle
    oracle.build()
    r = np.random.default_rng(20)
    hidden, heads, G, D, page, T = 256, 2, 2, 64, 32, 45
    N = (heads * G + 2 * heads) * D
    raw, raw_o = gen.weights_q8_0(N, hidden, seed=1, std=0.1), gen.weights_q4_0(hidden, heads * G * D, seed=2)
    wq = mmq.repack_weights("q8_0", torch.from_numpy(raw).cuda(), N, hidden)
    wo = mmq.repack_weights("q4_0", torch.from_numpy(raw_o).cuda(), hidden, heads * G * D)
    kc = torch.zeros(mmq.cache_shape("q8_0", 4, page, heads, D), dtype=torch.uint8, device="cuda")
    vc = torch.zeros(mmq.cache_shape("q4_0", 4, page, heads, D), dtype=torch.uint8, device="cuda")
    pages = r.permutation(4).astype(np.int32)
    table = torch.from_numpy(pages[None]).cuda()
    seen = 0
    for n in (T, 1, 1):                                    # a prompt, then two tokens
        x = r.standard_normal((n, hidden)).astype(np.float32)
        act = mmq.quantize_act(torch.from_numpy(x).cuda())
        qkv = mmq.gemm("q8_0", wq, act, n, N, hidden).view(n, -1, D)
        q, k, v = qkv[:, :heads * G], qkv[:, heads * G:heads * G + heads], qkv[:, heads * G + heads:]
        pos = seen + np.arange(n)
        slots = (pages[pos // page] * page + pos % page).astype(np.int32)
        mmq.cache_write(k, v, torch.from_numpy(slots).cuda(), kc, vc, vtype="q4_0")
        seen += n
        out = mmq.cache_attn(q, kc, vc, table, torch.tensor([seen], dtype=torch.int32, device="cuda"),
                             torch.tensor([0, n], dtype=torch.int32, device="cuda"), n, vtype="q4_0")
        y = mmq.gemm("q4_0", wo, mmq.quantize_act(out.view(n, -1)), n, hidden, heads * G * D)
        kv = [cachemodel.load(c.cpu().numpy(), t, s) for c, t, s in ((kc, "q8_0", "k"), (vc, "q4_0", "v"))]
        want, mag, terms = cachemodel.attn(q.cpu().numpy().astype(np.float64), *kv, pages[None], [seen], [0, n], page, 4, n,
                                           None, D ** -0.5)
        assert np.all(np.abs(out.cpu().numpy() - want) <= mag * 2e-4)      # coarse: the parts are tested alone
        rq, rs, _ = oracle.quantize_q8_1(out.cpu().numpy().reshape(n, -1))
        ref = oracle.gemm_f64("q4_0", raw_o, hidden, heads * G * D, rq, rs)
        assert np.max(np.abs(y.cpu().numpy() - ref)) <= 1e-3 * np.max(np.abs(ref))


def test_accepted_tokens_of_a_tree_are_written_to_their_places(env):
    """A tree is written behind the sequence; the accepted path's rows are written again, to the places
    that follow it, the others to none: the cache then reads as if only the path had been there."""
    torch, mmq = env
    heads, D, page = 2, 64, 32
    shape = mmq.cache_shape("q8_0", 3, page, heads, D)
    x = torch.randn(2, 60 + 8, heads, D, device="cuda")
    def slots(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")
    tree = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    mmq.cache_write(x[0], x[1], slots(list(range(68))), *tree)
    path = [0, 2, 5]
    to = [-1] * 8
    for j, p in enumerate(path):
        to[p] = 60 + j
    mmq.cache_write(x[0, 60:], x[1, 60:], slots(to), *tree)
    plain = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)]
    rows = list(range(60)) + [60 + p for p in path]
    mmq.cache_write(x[0][rows], x[1][rows], slots(list(range(63))), *plain)
    got, want = (mmq.cache_read(slots(list(range(63))), *c) for c in (tree, plain))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
def test_a_row_that_sees_one_token_gets_its_values(env, kind, dt):
    """One weight p, the same in the sum of weights and in the product. Its f16 terms are off by 2^-22 of it
    (bf16 rows, one term: 2^-11), and so are those of p times the scale; the product's two additions are
    off by 2^-23 each, the reciprocal and the last product by 2^-24 each: together 7 * 2^-23 of the
    value (2^-10 + 3 * 2^-23), and a bf16 result is rounded once more, by 2^-8."""
    torch, mmq = env
    c = Case(env, dt=dt, kt=kind, vt=kind, lens=(70, 1, 33), news=(5, 1, 3), tree=True, D=64, seed=13)
    c.lens[0], c.lens[2] = 5, 3                     # nothing but the new tokens
    c.mask[:] = [1 << i for i in (4, 3, 2, 1, 0, 0, 2, 2, 0)]
    got = c.device().run().float().cpu().numpy()
    v = cachemodel.load(c.host["v"], kind, "v").astype(np.float32)
    rel = 7 * 2.0 ** -23 if dt == "f32" else 2.0 ** -10 + 3 * 2.0 ** -23 + 2.0 ** -8
    for row, (b, pos) in enumerate([(0, 4), (0, 3), (0, 2), (0, 1), (0, 0), (1, 0), (2, 2), (2, 2), (2, 0)]):
        slot = c.table[b, pos // 32] * 32 + pos % 32
        want = v[slot].repeat(4, 0).astype(np.float64)
        assert np.all(np.abs(got[row] - want) <= rel * 1.01 * np.abs(want)), row


@pytest.mark.parametrize("n", [33, 777, 1900])
def test_equal_scores_give_the_mean(env, n):
    """q = 0: every weight is the same power of two, and whole numbers with scale 1 sum exactly; the quotient
    is off by two roundings."""
    torch, mmq = env
    c = Case(env, lens=(n,), news=(1,), D=64, page=64, seed=14)
    x = c.r.integers(-127, 128, (n, 2, 64)).astype(np.float32)
    x[:, :, ::32] = 127.0                           # every block's scale is 1
    slots = c.table[0, np.arange(n) // 64] * 64 + np.arange(n) % 64
    cachemodel.write(c.host["v"], x, slots, "q8_0", "v")
    c.device().q.zero_()
    got = c.run().cpu().numpy().astype(np.float64)[0]
    want = x.astype(np.float64).sum(0).repeat(4, 0) / n
    assert np.all(np.abs(got - want) <= np.abs(want) * 2 * U24 * 1.01)


@pytest.mark.parametrize("n", [40, 1500])
def test_a_query_that_is_not_a_number_gives_none(env, n):
    """And its neighbours, in the same products, are bit for bit what they are without it."""
    torch, mmq = env
    c = Case(env, lens=(n,), news=(3,), D=64, page=64, seed=15).device()
    before = c.run()
    c.q[1, 2, 5] = float("nan")
    after = c.run()
    assert torch.isnan(after[1, 2]).all()
    after[1, 2] = before[1, 2]
    assert torch.equal(after, before)


def _lens(n, low, high, seed):
    return tuple(int(x) for x in np.random.default_rng(seed).integers(low, high, n))


# many items and long tables: the work is one range that workgroups cut anywhere
CUT = [
    dict(lens=_lens(40, 1, 1500, 1), news=(1,) * 40, D=64, heads=4, page=64),
    dict(lens=_lens(12, 64, 1400, 2), news=_lens(12, 0, 21, 3), D=128, heads=8, G=2, dt="bf16", kt="q4_0", page=128),
    dict(lens=_lens(12, 64, 1400, 2), news=_lens(12, 0, 21, 3), D=128, heads=6, G=3, vt="q4_0", tree=True),
    dict(lens=_lens(9, 64, 1400, 4), news=_lens(9, 1, 65, 5), D=64, heads=3, G=2, dt="bf16", vt="q4_0", tree=True),
    dict(lens=(1200,), news=(400,), D=64, heads=2, G=4),
    dict(lens=(1200, 30, 950), news=(200, 30, 1), D=64, heads=2, G=4, dt="bf16", page=256),
    dict(lens=tuple((i * 37) % 97 + 900 * (i in (7, 500)) for i in range(600)), news=tuple(i % 3 for i in range(600)), D=64,
         heads=1, G=1),
    dict(lens=(1100, 1000), news=(2, 20), D=192, heads=8, G=2),
    dict(lens=(1100, 1000), news=(2, 20), D=256, heads=8, G=4, dt="bf16", kt="q4_0"),
    dict(lens=(1100, 1000), news=(2, 1), D=256, heads=1, vt="q4_0"),
    dict(lens=(1030,), news=(1,), D=192, heads=1, G=16, dt="bf16", kt="q4_0", vt="q4_0"),
    dict(lens=(40,), news=(3,), D=64, width=200),                          # a long table of a short sequence
]


@pytest.mark.parametrize("case", CUT, ids=lambda c: f"{len(c['lens'])}of{max(c['lens'])}-D{c['D']}-heads{c.get('heads', 2)}-{c.get('dt', 'f32')}")
def test_attention_cut_anywhere(env, case):
    test_attention(env, case)


def test_a_table_with_a_stride_and_an_unsigned_mask(env):
    torch, mmq = env
    c = Case(env, lens=(100, 64), news=(9, 12), tree=True, D=64, seed=16).device()
    want = c.check()
    wide = torch.full((2, c.width + 3), 7, dtype=torch.int32, device="cuda")
    wide[:, :c.width] = c.td
    c.td, c.md = wide[:, :c.width], c.md.view(torch.uint64)
    assert np.array_equal(c.run().cpu().numpy().astype(np.float64).reshape(want.shape), want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scales_that_are_negative(env, dt):
    """The quantiser makes none in q8_0, but a scale may have a sign: keys and values of both."""
    c = Case(env, dt=dt, lens=(150, 1000), news=(3, 1), D=64, page=64, seed=17)
    for side in "kv":
        rec = c.host[side]
        scales = rec[..., 64 * 32:].view(np.uint16)
        scales ^= (c.r.integers(0, 2, scales.shape) << 15).astype(np.uint16)
    c.device().check()


def test_a_cache_of_more_than_4_gib(env):
    """Pages below and above 2^32 bytes: what is written, read and attended to there is what a small cache
    with the same pages gives, and nothing else changes."""
    torch, mmq = env
    heads, D, page, G = 8, 256, 256, 2
    one = mmq.cache_bytes("q8_0", 1, page, heads, D)
    pages = 2 ** 32 // one + 40
    print(f"[case] cache of {pages} pages, {pages * one} bytes", flush=True)
    big = [torch.zeros(mmq.cache_shape("q8_0", pages, page, heads, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = [torch.zeros(mmq.cache_shape("q8_0", 5, page, heads, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    at = torch.tensor([pages - 1, 3, 2 ** 32 // one, pages - 7, 2 ** 31 // one], device="cuda")
    n = 5 * page - 11
    x = torch.randn(2, n, heads, D, device="cuda")
    pos = torch.arange(n, device="cuda")
    slots = (at[pos // page] * page + pos % page).int()
    for rows in (slice(0, 300), slice(300, n)):             # one by one, and windows of rows
        mmq.cache_write(x[0, rows], x[1, rows], slots[rows].clone(), *big)
        mmq.cache_write(x[0, rows], x[1, rows], pos[rows].int(), *small)
    for b, s in zip(big, small):
        assert torch.equal(b[at], s)
        b[at] = 0
        assert not b.view(torch.int64).any()
        b[at] = s
    for rows in (slice(0, 300), slice(0, n)):
        got, want = mmq.cache_read(slots[rows].clone(), *big), mmq.cache_read(pos[rows].int(), *small)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    q = torch.randn(20, heads * G, D, device="cuda")
    lens, starts = torch.tensor([n], dtype=torch.int32, device="cuda"), torch.tensor([0, 20], dtype=torch.int32, device="cuda")
    got = mmq.cache_attn(q, *big, at.int()[None], lens, starts, 20)
    want = mmq.cache_attn(q, *small, torch.arange(5, dtype=torch.int32, device="cuda")[None], lens, starts, 20)
    assert torch.equal(got, want)


def test_two_calls_at_once(env):
    """On two streams, each with a workspace of its own, and from two graphs: the bits of calls by themselves."""
    torch, mmq = env
    cases = [Case(env, lens=(3000, 1300), news=(1, 6), D=64, heads=4, page=64, seed=18).device(),
             Case(env, dt="bf16", lens=(2500, 700, 90), news=(7, 2, 30), D=128, page=64, seed=19).device()]
    want = [c.run() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, held = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(c.run())
        graphs.append(g)
    for turn in range(4):
        for h in held:
            h.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        got = []
        for _ in range(5):
            got = [c.run(stream=s) for c, s in zip(cases, streams)]
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for w, g, h in zip(want, got, held):
            assert torch.equal(w, g) and torch.equal(w, h)


@pytest.mark.parametrize("rows", [200, 2200])
def test_rows_written_and_read_in_a_graph(env, rows):
    """One by one and by windows: replayed with other rows and slots, as eager calls."""
    torch, mmq = env
    shape = mmq.cache_shape("q8_0", 80, 32, 8, 128)
    caches = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(4)]
    x = torch.zeros(2, rows, 8, 128, device="cuda")
    slots = torch.zeros(rows, dtype=torch.int32, device="cuda")
    back = torch.zeros(2, rows, 8, 128, device="cuda")
    def step(kc, vc, back):
        mmq.cache_write(x[0], x[1], slots, kc, vc)
        mmq.cache_read(slots, kc, vc, k=back[0], v=back[1])
    slots.copy_(torch.arange(rows))
    step(*caches[:2], back)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*caches[:2], back)
    caches[2].copy_(caches[0])
    caches[3].copy_(caches[1])
    for turn in range(4):
        x.copy_(torch.randn(x.shape, device="cuda"))
        slots.copy_(torch.arange(rows) + 7 * turn if turn % 2 else torch.randperm(80 * 32)[:rows])
        g.replay()
        want = torch.zeros_like(back)
        step(caches[2], caches[3], want)
        torch.cuda.synchronize()
        assert torch.equal(back, want) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_attention_refusals_of_the_binding(env):
    torch, mmq = env
    c = Case(env, lens=(70, 40), news=(2, 3), tree=True, D=64, seed=21).device()
    def refused(error, match, **kw):
        a = dict(q=c.q, kcache=c.kc, vcache=c.vc, table=c.td, lens=c.ld, starts=c.sd, max_q=c.max_q, mask=c.md)
        a.update(kw)
        with pytest.raises(error, match=match):
            mmq.cache_attn(**a)
    refused(ValueError, "mask", mask=c.md.int())
    refused(ValueError, "mask", mask=c.md[:4])
    refused(ValueError, "out", out=torch.empty(4, 8, 64, device="cuda"))
    refused(ValueError, "out", out=torch.empty(5, 8, 64, device="cuda", dtype=torch.bfloat16))
    refused(ValueError, "heads", q=c.q[:, :3])
    refused(ValueError, "q", q=c.q.transpose(1, 2))
    refused(ValueError, "rows", q=c.q.half())
    refused(ValueError, "table", table=c.td[0])
    refused(ValueError, "table", table=c.td.long())
    refused(ValueError, "table", table=c.td.t().contiguous().t())
    refused(ValueError, "table", lens=c.ld[:1])             # lens says how many sequences there are
    refused(ValueError, "starts", starts=c.sd[:2])
    refused(ValueError, "cache", kcache=c.kc[:, :, :, :-34])
    refused(ValueError, "cache", vcache=c.vc[:-1])
    refused(ValueError, "type", vtype="q5_0")
    refused(ValueError, "GPU", lens=c.ld.cpu())
    refused(mmq.MMQError, "mmq_cache_attn", max_q=0)
    refused(mmq.MMQError, "mmq_cache_attn", max_q=6)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        refused(mmq.MMQError, "mmq_cache_attn", scale=scale)
    wide = Case(env, lens=(1500,), news=(1,), D=64, seed=22).device()
    with pytest.raises(mmq.MMQError):
        wide.run(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def _put_values(c, slots, x):
    cachemodel.write(c.host["v"], x.astype(np.float32), slots, c.vt, "v")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,peak", [("q8_0", 2e3), ("q8_0", 1e5), ("q8_0", 1e6), ("q8_0", 8e6), ("q4_0", 200.0), ("q4_0", 5e5)])
@pytest.mark.parametrize("where", ["block", "before", "tree", "chain"])
def test_a_large_value_scale_leaves_the_others_their_bits(env, where, kind, peak, dt):
    """A row that sees one token (of weight 1; what else it sees is 2^-200 of it), with a block of values of `peak`
    in that token, in a token before it that the same wave has had, or in one of the same tile that the row
    does not see. Relative: as in test_a_row_that_sees_one_token_gets_its_values. Absolute: the products' f16 terms are
    held to 2^-25 where the row's largest weight, times its token's scale over 4 where that is above one, is
    at least 2^8, so 2^-33 max(1, D / 4) of a whole number q, with D the largest scale of the token it sees."""
    torch, mmq = env
    if where == "before":                       # tiles 0 and 4 are one wave's
        c = Case(env, dt=dt, vt=kind, lens=(129,), news=(1,), D=64, seed=31)
        k = np.full((129, 2, 64), -4.0, np.float32)
        k[128] = 4.0
        slots = c.table[0, np.arange(129) // 32] * 32 + np.arange(129) % 32
        cachemodel.write(c.host["k"], k, slots, "q8_0", "k")
        c.qh[:] = 4.0                           # scores -128 and 128
        rows, large = [(0, 128)], 5
    elif where == "chain":                      # row 0 sees token 0 alone
        c = Case(env, dt=dt, vt=kind, lens=(20,), news=(20,), D=64, seed=32)
        rows, large = [(0, 0)], 7
    else:
        c = Case(env, dt=dt, vt=kind, lens=(20,), news=(20,), tree=True, D=64, seed=33)
        c.mask[:] = [1 << i for i in range(20)]
        large = 7
        rows = [(i, i) for i in range(20) if (i == large) == (where == "block")]
    n = int(c.lens[0])
    slots = c.table[0, np.arange(n) // 32] * 32 + np.arange(n) % 32
    x = c.r.uniform(-3, 3, (n, 2, 64))
    x[large, :, :32] *= peak / 3
    x[large, :, 0] = peak
    _put_values(c, slots, x)
    got = c.device().run().float().cpu().numpy().astype(np.float64)
    values = cachemodel.load(c.host["v"], kind, "v")
    q, top = (127, 254.0) if kind == "q8_0" else (8, 16.0)
    rel = 7 * 2.0 ** -23 if dt == "f32" else 2.0 ** -10 + 3 * 2.0 ** -23 + 2.0 ** -8
    for row, pos in rows:
        want = values[slots[pos]].repeat(4, 0)
        D = np.abs(want).max() / (top / 2)
        off = np.abs(got[row] - want) - rel * 1.01 * np.abs(want)
        assert np.all(off <= q * 2.0 ** -33 * max(1.0, D / 4) * 1.01), (row, off.max())


def _as_held(c):
    """Case.want() with its absolute term, N 2^-28 max|v|, as the products' terms have it: p's are held to 2^-25 where
    the largest weight is 2^8, and p d 2^k's to 2^-25 where the largest weight times 4 (or times 2^15 of a scale, k
    being at most 15) is 2^8, so to N (2^-33 + 2^-35) max|v| + N 127 2^-48. There are two roundings of a term, the
    second 2^-21 in f32 rows: of the two numbers of 2^-11 that are added."""
    want, bound = c.want()
    k, v = (cachemodel.load(c.host[s], t, s) for s, t in (("k", c.kt), ("v", c.vt)))
    with np.errstate(invalid="ignore"):
        mag = cachemodel.attn(c.qh.astype(np.float64), k, v, c.table, c.lens, c.starts, c.page, c.pages, c.max_q, c.mask, c.scale)[1]
    used = np.concatenate([c.table[b, np.arange(n) // c.page] * c.page + np.arange(n) % c.page for b, n in enumerate(c.lens)])
    vmax, N = np.abs(v[used]).max(), int(c.lens.max())
    bound += N * ((2.0 ** -33 + 2.0 ** -35 - 2.0 ** -28) * vmax + 127 * 2.0 ** -48)
    return want, bound + mag * (2.0 ** -21 if c.dt == "f32" else 2.0 ** -11) * 1.01


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("std", [1e-3, 1.0, 1e3, 3e4])
def test_attention_within_the_absolute_bound_of_its_terms(env, std, kind, dt):
    """Values of one size, large scales from 1e3 on (1e2 in q4_0)."""
    torch, mmq = env
    c = Case(env, dt=dt, vt=kind, lens=(200, 450, 31), news=(2, 5, 1), D=64, seed=35)
    for b, n in enumerate(c.lens):
        slots = c.table[b, np.arange(n) // 32] * 32 + np.arange(n) % 32
        x = c.r.standard_normal((n, 2, 64)) * std
        x[::7] *= 3
        _put_values(c, slots, x)
    got = c.device().run().float().cpu().numpy().astype(np.float64)
    want, bound = _as_held(c)
    off = np.abs(got - want)
    print(f"[case]   error at most {(off / bound).max():.4f} of the bound", flush=True)
    assert np.all(off <= bound)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("n,news,D,kind", [(300, 1, 64, "q8_0"), (640, 5, 128, "q4_0"), (1900, 1, 64, "q8_0"), (900, 12, 128, "q8_0"),
                                           (500, 3, 192, "q4_0"), (700, 2, 256, "q8_0")])
def test_equal_scores_over_scales_of_all_sizes(env, n, news, D, kind, dt):
    """q = 0, and blocks of values from 1e-3 to 1e6 (1e5 in q4_0) beside and after each other, the last one
    ordinary. Weights are 1 / N, so what the terms do not hold, N (2^-33 + 2^-35) max|v| of the largest weight,
    is 1.25 2^-33 max|v| here."""
    torch, mmq = env
    c = Case(env, dt=dt, vt=kind, lens=(n,), news=(news,), D=D, page=64, seed=36)
    c.qh[:] = 0
    slots = c.table[0, np.arange(n) // 64] * 64 + np.arange(n) % 64
    size = 10.0 ** c.r.uniform(-3, 6 if kind == "q8_0" else 5, (n, 2, D // 32, 1))
    size[c.r.random(n) < 0.7] = 1.0
    size[:, :, -1] = 1.0                            # a block of ordinary values in every token
    _put_values(c, slots, (c.r.standard_normal((n, 2, D // 32, 32)) * size).reshape(n, 2, D))
    got = c.device().run().float().cpu().numpy().astype(np.float64)
    v = cachemodel.load(c.host["v"], kind, "v")[slots]
    for i in range(news):
        seen = v[:n - news + i + 1]
        want, mag = seen.mean(0).repeat(4, 0), np.abs(seen).mean(0).repeat(4, 0)
        # sums over n + 32 additions, weights that are powers of two exactly; terms of 2^-22 and 2^-21, or 2^-11 twice
        bound = mag * (4 * U24 * (n + 32) + (3 * 2.0 ** -22 if dt == "f32" else 2.0 ** -10)) * 1.01 + 1.25 * 2.0 ** -33 * np.abs(seen).max()
        bound += np.abs(want) * (U24 if dt == "f32" else 2.0 ** -8)
        off = np.abs(got[i] - want)
        print(f"[case]   error at most {(off / bound).max():.4f} of the bound", flush=True)
        assert np.all(off <= bound)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_large_and_infinite_scales_in_one_tile(env, dt):
    """Each row sees its own token, one of them with values up to 1e6, one with infinite scales (head 0), which row 5
    sees besides its own: rows of the infinite one are not finite, all others as if they were alone."""
    torch, mmq = env
    c = Case(env, dt=dt, lens=(20,), news=(20,), tree=True, D=64, seed=37)
    c.mask[:] = [1 << i for i in range(20)]
    c.mask[5] |= np.uint64(1 << 3)
    slots = c.table[0, np.arange(20) // 32] * 32 + np.arange(20) % 32
    x = c.r.uniform(-3, 3, (20, 2, 64))
    x[2, :, 7] = 1e6
    _put_values(c, slots, x)
    values = cachemodel.load(c.host["v"], "q8_0", "v")[slots]
    t = int(slots[3]) % 32
    for b in range(2):
        at = 64 * 32 + 2 * (((t % 16) // 4 * 2 + b) * 8 + 4 * (t // 16) + t % 4)
        c.host["v"][slots[3] // 32, 0, 0, at:at + 2] = np.frombuffer(np.uint16(0x7C00).tobytes(), np.uint8)
    got = c.device().run().float().cpu().numpy().astype(np.float64)
    assert not np.isfinite(got[[3, 5], :4]).any() and np.isfinite(got[[3, 5], 4:]).all()
    rel = 7 * 2.0 ** -23 if dt == "f32" else 2.0 ** -10 + 3 * 2.0 ** -23 + 2.0 ** -8
    for row in (i for i in range(20) if i not in (3, 5)):
        want = values[row].repeat(4, 0)
        D = np.abs(want).max() / 127
        assert np.all(np.abs(got[row] - want) <= rel * 1.01 * np.abs(want) + 127 * 2.0 ** -33 * max(1.0, D / 4) * 1.01), row


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,news,n", [(64, 3, 700), (128, 8, 650), (256, 3, 700)])
def test_a_row_keeps_its_bits_whatever_its_neighbours_are(env, D, news, n, dt):
    """Several tiles a wave, so that running maxima are taken anew: a neighbour in the same products whose scores
    rise along the sequence, are not numbers, or are all alike, and the other rows bit for bit the same."""
    torch, mmq = env
    c = Case(env, dt=dt, lens=(n,), news=(news,), D=D, page=64, seed=34)
    slots = c.table[0, np.arange(n) // 64] * 64 + np.arange(n) % 64
    k = c.r.standard_normal((n, 2, D)).astype(np.float32)
    k[:, :, 7] = np.linspace(0, 4, n)[:, None]
    cachemodel.write(c.host["k"], k, slots, "q8_0", "k")
    c.device().q[:, :, 7] = 0.0
    runs = []
    for neighbour in (0.0, 200.0, float("nan")):
        c.q[1, 2] = 0.0
        c.q[1, 2, 7] = neighbour
        runs.append(c.run())
    assert torch.isnan(runs[2][1, 2]).all()
    for got in runs[1:]:
        got[1, 2] = runs[0][1, 2]
        assert torch.equal(got, runs[0])


# items cut anywhere whose join has several rows a workgroup, for heads whose rows do not fill one (192) and for those
# of one wave a SIMD (256, more than 32 items)
CUT_WIDE = [
    dict(lens=_lens(12, 64, 1400, 6), news=_lens(12, 1, 21, 7), D=192, heads=8, G=2),
    dict(lens=_lens(12, 64, 1400, 6), news=_lens(12, 1, 21, 7), D=192, heads=8, G=2, dt="bf16", kt="q4_0", page=128),
    dict(lens=_lens(9, 64, 1400, 8), news=_lens(9, 1, 30, 9), D=192, heads=6, G=3, vt="q4_0", tree=True),
    dict(lens=(1100, 1000), news=(2, 20), D=256, heads=8, G=4),
    dict(lens=_lens(12, 64, 1400, 10), news=(1,) * 12, D=256, heads=4, G=3, vt="q4_0"),
]


@pytest.mark.parametrize("case", CUT_WIDE, ids=lambda c: f"{len(c['lens'])}of{max(c['lens'])}-D{c['D']}-heads{c.get('heads', 2)}-{c.get('dt', 'f32')}")
def test_attention_cut_anywhere_in_wide_heads(env, case):
    test_attention(env, case)


@pytest.mark.parametrize("case", [
    dict(lens=(20011, 9000), news=(1, 3), D=64, heads=1, G=2, page=256),
    dict(lens=(33000,), news=(2,), D=128, heads=1, G=1, page=64, dt="bf16", vt="q4_0"),
    dict(lens=_lens(36, 4000, 9000, 11), news=(1,) * 36, D=64, heads=2, G=1, kt="q4_0"),
], ids=lambda c: f"{len(c['lens'])}of{max(c['lens'])}")
def test_attention_over_long_sequences(env, case):
    c = Case(env, **case).device()
    want, bound = _as_held(c)
    off = np.abs(c.run().float().cpu().numpy().astype(np.float64) - want)
    print(f"[case]   error at most {(off / bound).max():.4f} of the bound", flush=True)
    assert np.all(off <= bound)


@pytest.mark.parametrize("n,news,kind", [(33001, 1, "q8_0"), (131071, 1, "q4_0"), (16385, 5, "q8_0")])
def test_equal_scores_give_the_mean_of_long_sequences(env, n, news, kind):
    """As test_equal_scores_give_the_mean: whole numbers below 2^24 in all, so every token counts, or the sum is off."""
    torch, mmq = env
    c = Case(env, vt=kind, lens=(n,), news=(news,), D=64, page=128, seed=38)
    top = 127 if kind == "q8_0" else 7
    x = c.r.integers(-top, top + 1, (n, 2, 64)).astype(np.float32)
    x[:, :, ::32] = 127.0 if kind == "q8_0" else -8.0          # every block's scale is 1
    slots = c.table[0, np.arange(n) // 128] * 128 + np.arange(n) % 128
    cachemodel.write(c.host["v"], x, slots, kind, "v")
    c.device().q.zero_()
    got = c.run().cpu().numpy().astype(np.float64)
    for i in range(news):
        seen = n - news + i + 1
        want = x[:seen].astype(np.float64).sum(0).repeat(4, 0) / seen
        assert np.all(np.abs(got[i] - want) <= np.abs(want) * 2 * U24 * 1.01)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [9, 1700])
def test_rows_of_odd_strides(env, dt, rows):
    """Queries, keys and values whose rows lie an odd number of elements apart: the bits of contiguous ones."""
    torch, mmq = env
    heads, D, page, dtype = 8, 128, 64, _dtype(torch, dt)
    x = torch.randn(3, rows, heads * D, device="cuda").to(dtype)
    q, k, v = (torch.zeros(rows * (heads * D + s) + 8, dtype=dtype, device="cuda")[:rows * (heads * D + s)].view(rows, -1)[:, :heads * D]
               for s in (1, 3, 5))
    for to, of in zip((q, k, v), x):
        to.copy_(of)
    shape = mmq.cache_shape("q8_0", rows // page + 2, page, heads, D)
    slots = torch.arange(5, 5 + rows, dtype=torch.int32, device="cuda")
    caches = [torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(4)]
    mmq.cache_write(k, v, slots, caches[0], caches[1])
    mmq.cache_write(x[1], x[2], slots, caches[2], caches[3])
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    table = torch.arange(rows // page + 2, dtype=torch.int32, device="cuda")[None]
    lens, starts = (torch.tensor(n, dtype=torch.int32, device="cuda") for n in ([5 + rows], [0, 9]))
    got, want = (mmq.cache_attn(t[:9], caches[0], caches[1], table, lens, starts, 9) for t in (q, x[0]))
    assert q.stride(0) % 2 == 1 and torch.equal(got, want)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,kind", [(64, "q8_0"), (128, "q4_0"), (192, "q8_0")])
def test_small_scores_over_large_scales(env, D, kind, dt):
    """Weights of all sorts near 1 / N times scales from 8 on, with scores so small that the bound is a few 2^-16: of
    some 100000 products of a weight and a scale, each has its two terms."""
    torch, mmq = env
    c = Case(env, dt=dt, vt=kind, lens=(64,), news=(64,), D=D, heads=2, G=8, seed=39)
    c.qh *= np.float32(2.0 ** -6)
    slots = c.table[0, np.arange(64) // 32] * 32 + np.arange(64) % 32
    size = 10.0 ** c.r.uniform(2, 6 if kind == "q8_0" else 4.9, (64, 2, D // 32, 1))
    _put_values(c, slots, (c.r.standard_normal((64, 2, D // 32, 32)) * size).reshape(64, 2, D))
    got = c.device().run().float().cpu().numpy().astype(np.float64)
    want, bound = _as_held(c)
    off = np.abs(got - want)
    print(f"[case]   error at most {(off / bound).max():.4f} of the bound", flush=True)
    assert np.all(off <= bound)
