"""Host-side tests of the key/value cache calls (no GPU needed): sizes, the refusals, each of which
returns before any HIP call, the binding's own checks, and the layout's addresses."""
import ctypes

import numpy as np
import pytest

import cachemodel


@pytest.fixture(scope="module")
def mmq():
    import os
    import block_quantized_int8_amd as m
    if not os.path.exists(m.LIB_PATH):
        from block_quantized_int8_amd import build
        build.build()
    m.lib()
    return m


BAD, GOOD = ctypes.c_void_p(0x1001), ctypes.c_void_p(0x10000)     # never dereferenced
Q8, Q4 = 0, 1


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("kind,rec", [("q8_0", 34), ("q4_0", 18)])
def test_cache_sizes(mmq, kind, rec, page, D):
    assert mmq.cache_bytes(kind, 7, page, 3, D) == 7 * page * 3 * D // 32 * rec
    assert mmq.cache_shape(kind, 7, page, 3, D) == (7, 3, page // 32, rec * D)


@pytest.mark.parametrize("args", [(Q8, 0, 32, 1, 64), (Q8, -1, 32, 1, 64), (Q8, 1, 16, 1, 64), (Q8, 1, 48, 1, 64),
                                  (Q8, 1, 512, 1, 64), (Q8, 1, 32, 0, 64), (Q8, 1, 32, 1025, 64), (Q8, 1, 32, 1, 0),
                                  (Q8, 1, 32, 1, 32), (Q8, 1, 32, 1, 96), (Q8, 1, 32, 1, 320), (2, 1, 32, 1, 64),
                                  (99, 1, 32, 1, 64), (-1, 1, 32, 1, 64), (Q4, 1 << 26, 32, 1, 64), (Q4, 1 << 62, 256, 1, 64)])
def test_cache_sizes_refused(mmq, args):
    assert mmq.lib().mmq_cache_bytes(*args) == 0
    with pytest.raises(mmq.MMQError):
        mmq.cache_shape(*args)


def test_the_largest_cache(mmq):
    assert mmq.cache_bytes("q8_0", (1 << 26) - 1, 32, 8, 128) == ((1 << 26) - 1) * 8 * 4352


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("side", ["k", "v"])
def test_the_layout_holds_every_value_once(kind, side):
    """Each value of a record has bits of its own, and all of the record's are taken."""
    D = 192
    rec = np.zeros(cachemodel.BLOCK[kind] * D, np.int64)
    for t in range(32):
        one = np.zeros(rec.size, np.uint8)
        full = np.full((D // 32, 32), 127 if kind == "q8_0" else 7)
        scale = np.full(D // 32, -1, np.int16).view(np.float16)
        cachemodel.store(one, t, full, scale, kind, side)
        assert np.all((rec & one) == 0)
        rec |= one
    assert np.all(rec == 255)


@pytest.mark.parametrize("kind", ["q8_0", "q4_0"])
@pytest.mark.parametrize("side", ["k", "v"])
def test_the_model_reads_what_it_writes(kind, side):
    r = np.random.default_rng(3)
    cache = r.integers(0, 256, (3, 2, 2, cachemodel.BLOCK[kind] * 64)).astype(np.uint8)
    x = r.standard_normal((100, 2, 64)).astype(np.float32)
    slots = r.permutation(3 * 64)[:100]
    cachemodel.write(cache, x, slots, kind, side)
    got = cachemodel.load(cache, kind, side)[slots]
    assert np.array_equal(got, cachemodel.value_of(*cachemodel.quantize(x, kind)))
    one = np.zeros_like(cache)                              # and writes what store() does, one by one
    all_ = np.zeros_like(cache)
    q, d = cachemodel.quantize(x, kind)
    for row, slot in enumerate(slots):
        for h in range(2):
            cachemodel.store(one[slot // 64, h, slot // 32 % 2], slot % 32, q[row, h], d[row, h], kind, side)
    cachemodel.write(all_, x, slots, kind, side)
    assert np.array_equal(one, all_)


def _calls(mmq):
    L = mmq.lib()

    def write(o=0, k=GOOD, ldk=512, v=GOOD, ldv=512, slots=GOOD, rows=5, tk=Q8, kcache=GOOD, tv=Q4, vcache=GOOD, pages=4,
              page=64, heads=4, D=128):
        return L.mmq_cache_write(o, k, ldk, v, ldv, slots, rows, tk, kcache, tv, vcache, pages, page, heads, D, None)

    def read(o=0, k=GOOD, ldk=512, v=GOOD, ldv=512, slots=GOOD, rows=5, tk=Q8, kcache=GOOD, tv=Q4, vcache=GOOD, pages=4,
             page=64, heads=4, D=128):
        return L.mmq_cache_read(o, slots, rows, tk, kcache, tv, vcache, pages, page, heads, D, k, ldk, v, ldv, None)

    def attn(o=0, q=GOOD, ldq=1024, rows=5, heads_q=8, tk=Q8, kcache=GOOD, tv=Q4, vcache=GOOD, pages=4, page=64, heads=4,
             D=128, table=GOOD, ldt=100, width=100, lens=GOOD, starts=GOOD, B=2, max_q=3, mask=None, scale=0.1, out=GOOD,
             ldo=1024, workspace=GOOD, ws=1 << 40):
        return L.mmq_cache_attn(o, q, ldq, rows, heads_q, tk, kcache, tv, vcache, pages, page, heads, D, table, ldt, width,
                                lens, starts, B, max_q, mask, scale, out, ldo, workspace, ws, None)
    return write, read, attn


def test_row_call_refusals(mmq):
    write, read, attn = _calls(mmq)
    for f in (write, read, attn):
        for pages, page, heads, D in ((0, 64, 4, 128), (4, 16, 4, 128), (4, 96, 4, 128), (4, 64, 0, 128), (4, 64, 4, 96),
                                      (1 << 25, 64, 4, 128), (-3, 64, 4, 128)):
            assert f(pages=pages, page=page, heads=heads, D=D) == mmq.MMQ_EINVAL
        for kw in ({"o": 3}, {"o": -1}, {"tk": 8}, {"tv": -1}, {"rows": 0}, {"rows": (1 << 24) + 1}):
            assert f(**kw) == mmq.MMQ_EINVAL, kw
        for kw in ({"o": 2}, {"tk": 2}, {"tv": 4}, {"tk": 6}):
            assert f(**kw) == mmq.MMQ_EUNSUPPORTED, kw
    for f in (write, read):
        for p in ("k", "v", "slots", "kcache", "vcache"):
            assert f(**{p: None}) == mmq.MMQ_EINVAL, p
            assert f(**{p: BAD}) == mmq.MMQ_EALIGN, p
        for ld in ("ldk", "ldv"):
            assert f(**{ld: 511}) == mmq.MMQ_EINVAL, ld
        assert f(rows=1 << 24, heads=1024, D=128, ldk=1 << 20, ldv=1 << 20) == mmq.MMQ_EINVAL


def test_attn_refusals(mmq):
    attn = _calls(mmq)[2]
    for p in ("q", "kcache", "vcache", "table", "lens", "starts", "out"):
        assert attn(**{p: None}) == mmq.MMQ_EINVAL, p
        assert attn(**{p: BAD}) == mmq.MMQ_EALIGN, p
    assert attn(mask=BAD) == mmq.MMQ_EALIGN
    for kw in ({"ldq": 1023}, {"ldo": 1023}, {"ldt": 99}, {"width": 0}, {"width": (1 << 22) + 1, "ldt": 1 << 23}, {"B": 0},
               {"B": 4097}, {"max_q": 0}, {"max_q": 6}, {"heads_q": 6}, {"heads_q": 0}, {"heads_q": 2},
               {"heads_q": 4100, "ldq": 1 << 20, "ldo": 1 << 20}, {"scale": 0.0}, {"scale": -1.0}, {"scale": float("nan")},
               {"scale": float("inf")}, {"mask": GOOD, "rows": 65, "max_q": 65}):
        assert attn(**kw) == mmq.MMQ_EINVAL, kw
    big = dict(rows=1 << 24, max_q=1 << 24, heads_q=8)
    assert attn(**big) == mmq.MMQ_EINVAL                    # too many groups of rows for a launch
    need = mmq.cache_attn_workspace_bytes(5, 8, 64, 4, 128, 100, 2, 3)
    assert need > 0
    assert attn(workspace=None) == mmq.MMQ_EWORKSPACE
    assert attn(ws=need - 1) == mmq.MMQ_EWORKSPACE
    assert attn(workspace=BAD) == mmq.MMQ_EALIGN


def test_attn_workspace_sizes(mmq):
    f = mmq.cache_attn_workspace_bytes
    assert f(1, 8, 32, 4, 128, 1, 1, 1) == 0                # one launch
    for bad in ((0, 8, 32, 4, 128, 1, 1, 1), (1, 7, 32, 4, 128, 1, 1, 1), (1, 8, 16, 4, 128, 1, 1, 1),
                (1, 8, 32, 4, 100, 1, 1, 1), (1, 8, 32, 4, 128, 0, 1, 1), (1, 8, 32, 4, 128, 1, 0, 1),
                (1, 8, 32, 4, 128, 1, 1, 2)):
        assert f(*bad) == 0
    # bounded by the card, not by the batch: a chunk's sums are kept for split sequences alone
    assert 0 < f(4096, 32, 64, 8, 128, 4096, 4096, 1) < 64 << 20
    assert 0 < f(4096, 1024, 64, 1024, 256, 4096, 64, 64) < 1 << 30


def test_binding_refuses(mmq):
    import torch
    cache = torch.zeros(mmq.cache_shape("q8_0", 2, 64, 4, 128), dtype=torch.uint8)
    slots = torch.zeros(5, dtype=torch.int32)
    rows = torch.zeros(5, 4, 128)
    with pytest.raises(ValueError, match="GPU"):
        mmq.cache_write(rows, rows, slots, cache, cache)
    with pytest.raises(ValueError, match="GPU"):
        mmq.cache_read(slots, cache, cache)
    with pytest.raises(ValueError, match="GPU"):
        mmq.cache_attn(rows, cache, cache, slots.view(1, 5), slots[:1], slots[:2], 1)
    f = "f"
    for kt, vt in (("q8_1", "q8_0"), ("q8_0", 0), (None, "q4_0")):
        with pytest.raises(ValueError, match="type"):
            mmq._caches(f, cache, cache, kt, vt)
    for k, v in ((cache, cache[:1]), (cache, cache.view(torch.int8)), (cache[:, :, :, :-1], cache), (cache.view(-1), cache),
                 (cache, torch.zeros(mmq.cache_shape("q4_0", 2, 64, 4, 128), dtype=torch.uint8))):
        with pytest.raises(ValueError):
            mmq._caches(f, k, v, "q8_0", "q8_0")
    assert mmq._caches(f, cache, torch.zeros(mmq.cache_shape("q4_0", 2, 64, 4, 128), dtype=torch.uint8), "q8_0", "q4_0") \
        == (0, 1, 2, 64, 4, 128)


def test_binding_strides(mmq):
    import torch
    f32 = torch.float32
    x = torch.zeros(5, 12, 64)
    assert mmq._heads_ld("f", "k", x, 12, 64, f32) == (5, 768)
    assert mmq._heads_ld("f", "k", x[:, 4:8], 4, 64, f32) == (5, 768)
    assert mmq._heads_ld("f", "k", x.view(5, 768), 12, 64, f32) == (5, 768)
    assert mmq._heads_ld("f", "k", x[:1, 2:3], 1, 64, f32) == (1, 768)
    assert mmq._heads_ld("f", "k", x.transpose(0, 1)[:1, :, :].transpose(0, 1), 1, 64, f32) == (5, 768)
    for t in (x.transpose(0, 1), x[:, ::2], x[:, :, ::2], x.double(), x[0], x[:, :, :63]):
        with pytest.raises(ValueError):
            mmq._heads_ld("f", "k", t, 12, 64, f32)


def test_caches_without_heads_or_values_are_refused(mmq):
    """A ValueError as for other shapes, before anything is divided by them."""
    import torch
    for shape in ((2, 0, 2, 34 * 64), (2, 4, 2, 0), (2, 0, 2, 0)):
        cache = torch.zeros(shape, dtype=torch.uint8)
        with pytest.raises(ValueError, match="cache_shape"):
            mmq._caches("f", cache, cache, "q8_0", "q8_0")
