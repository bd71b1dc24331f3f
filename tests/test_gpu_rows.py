"""Rows grouped by expert on the GPU, through the public binding: the plan against a numpy sort,
the gather bit for bit, the combination and its gradients against 64-bit sums.

Tolerances. An f32 sum of k products, fused multiply-adds in any order, is off by at most
k * 2^-24 * sum |terms| (first order; 1.01 covers the rest); a value rounded once to bf16 by at
most 2^-8 of itself, on top."""
import numpy as np
import pytest

import rowmodel

pytestmark = pytest.mark.gpu

U24, U8 = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def env():
    import torch
    import block_quantized_int8_amd as mmq
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mmq.lib()
    return torch, mmq


def _ids(T, top_k, E, away, seed, wild=False):
    r = np.random.default_rng([seed, T, top_k, E])
    ids = np.argsort(r.random((T, E)), axis=1)[:, :top_k].astype(np.int32) if E <= 512 else \
        r.integers(0, E, (T, top_k)).astype(np.int32)
    if wild:                                # the same expert twice, and ids far outside the range
        ids[:, -1] = ids[:, 0]
        ids[r.random(ids.shape) < 0.1] = np.iinfo(np.int32).max
        ids[r.random(ids.shape) < 0.1] = np.iinfo(np.int32).min
        ids[r.random(ids.shape) < 0.1] = E
    ids[r.random(ids.shape) < away] = -1
    return ids


PLANS = [(1, 1, 1, 0.0), (1, 1, 1, 1.0), (7, 1, 3, 0.3), (64, 1, 1, 0.0), (65, 1, 1, 0.0), (10, 8, 64, 0.0),
         (513, 3, 5, 0.5), (300, 17, 33, 0.1), (1025, 2, 1023, 0.0), (777, 2, 1024, 0.2), (900, 5, 4096, 0.1),
         (32768, 1, 9, 0.1), (32769, 1, 9, 0.1), (20001, 4, 130, 0.0), (70000, 1, 1, 0.0), (11003, 3, 2000, 0.3)]


@pytest.mark.parametrize("T,top_k,E,away", PLANS)
def test_plan_is_the_stable_sort(env, T, top_k, E, away):
    torch, mmq = env
    print(f"[case] plan T={T} top_k={top_k} E={E} away={away}", flush=True)
    ids = _ids(T, top_k, E, away, 1, wild=T % 3 == 0)
    plan = torch.full((mmq.group_bytes(E, T, top_k),), 0xA5, dtype=torch.uint8, device="cuda")
    mmq.group_rows(torch.from_numpy(ids).cuda(), E, out=plan)
    got = [v.cpu().numpy() for v in mmq.group_views(plan, E, T, top_k)]
    for name, g, w in zip(("offs", "order", "pos", "units"), got, rowmodel.plan(ids, E)):
        assert np.array_equal(g, w), name


def _dtype(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _host(t):
    return t.float().cpu().numpy().astype(np.float64)


def _strided(torch, rows, N, ld, dt, fill, seed):
    """[rows, N] inside a [rows, ld] buffer, random values over a filled frame."""
    buf = torch.full((rows, ld), fill, dtype=dt, device="cuda")
    g = torch.Generator().manual_seed(seed)
    buf[:, :N] = torch.randn((rows, N), generator=g).to(dt).cuda()
    return buf, buf[:, :N]


ROWS = [("f32", 1, 1, 1, 1, 1, 0.0), ("bf16", 1, 1, 1, 1, 1, 0.0), ("bf16", 5, 2, 3, 7, 7, 0.2),
        ("f32", 3, 3, 4, 3, 5, 0.3), ("bf16", 9, 4, 8, 1001, 1001, 0.25), ("f32", 33, 8, 64, 1030, 1031, 0.0),
        ("bf16", 40, 9, 16, 2052, 2060, 0.5), ("f32", 20, 17, 33, 260, 260, 0.1), ("f32", 130, 4, 8, 4096, 4096, 1.0),
        ("bf16", 1100, 4, 8, 520, 521, 0.5), ("f32", 1030, 5, 8, 90, 91, 0.1), ("f32", 66000, 1, 2, 5, 5, 0.1)]


@pytest.mark.parametrize("dt,T,top_k,E,N,ld,away", ROWS)
def test_gather(env, dt, T, top_k, E, N, ld, away):
    torch, mmq = env
    print(f"[case] gather {dt} T={T} top_k={top_k} E={E} N={N} ld={ld}", flush=True)
    ids = _ids(T, top_k, E, away, 2, wild=top_k > 2)
    _, x = _strided(torch, T, N, ld, _dtype(torch, dt), 3.0, 5)
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    buf = torch.full((T * top_k, ld + 3), -7.0, dtype=x.dtype, device="cuda")
    mmq.moe_gather(x, plan, E, top_k, out=buf[:, :N])
    want = np.full((T * top_k, ld + 3), -7.0)
    row = rowmodel.row_of(ids, E, "sorted")
    t, j = np.nonzero(row >= 0)
    want[row[t, j], :N] = _host(x)[t]
    assert np.array_equal(_host(buf), want)


@pytest.mark.parametrize("order", ["pair", "sorted"])
@pytest.mark.parametrize("dt,T,top_k,E,N,ld,away", ROWS)
def test_combine(env, dt, T, top_k, E, N, ld, away, order):
    torch, mmq = env
    print(f"[case] combine {dt} {order} T={T} top_k={top_k} E={E} N={N} ld={ld}", flush=True)
    ids = _ids(T, top_k, E, away, 3, wild=top_k > 2)
    row = rowmodel.row_of(ids, E, order)
    zb, z = _strided(torch, T * top_k, N, ld, _dtype(torch, dt), 3.0, 6)
    used = np.zeros(T * top_k, bool)
    used[row[row >= 0]] = True
    z[torch.from_numpy(~used).cuda()] = float("nan")          # rows of no pair: never read
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    w = np.random.default_rng(4).standard_normal((T, top_k)).astype(np.float32)
    w[row < 0] = np.nan                                       # nor their weights' values used
    zh = np.where(used[:, None], _host(z), 0.0)
    for weights in (w, None):
        wh = np.where(row >= 0, 1.0 if weights is None else weights, 0.0).astype(np.float64)
        terms = wh[:, :, None] * zh[np.maximum(row, 0)]
        want, bound = terms.sum(1), np.abs(terms).sum(1) * top_k * U24 * 1.01
        if dt == "bf16":
            bound += (np.abs(want) + bound) * U8
        buf = torch.full((T, ld + 1), -7.0, dtype=z.dtype, device="cuda")
        mmq.moe_combine(z, plan, E, T, top_k, weights=None if weights is None else torch.from_numpy(w).cuda(),
                        order=order, out=buf[:, :N])
        got = _host(buf)
        assert np.all(got[:, N:] == -7.0)
        assert np.all(np.abs(got[:, :N] - want) <= bound)
        assert np.all(got[(row < 0).all(1), :N] == 0.0)


@pytest.mark.parametrize("order", ["pair", "sorted"])
@pytest.mark.parametrize("dt,T,top_k,E,N,ld,away", ROWS)
def test_combine_grad(env, dt, T, top_k, E, N, ld, away, order):
    torch, mmq = env
    print(f"[case] combine_grad {dt} {order} T={T} top_k={top_k} E={E} N={N} ld={ld}", flush=True)
    ids = _ids(T, top_k, E, away, 7, wild=top_k > 2)
    row = rowmodel.row_of(ids, E, order)
    _, z = _strided(torch, T * top_k, N, ld, _dtype(torch, dt), 3.0, 8)
    used = np.zeros(T * top_k, bool)
    used[row[row >= 0]] = True
    z[torch.from_numpy(~used).cuda()] = float("nan")
    _, dy = _strided(torch, T, N, ld + 2, _dtype(torch, dt), 3.0, 9)
    w = np.random.default_rng(5).standard_normal((T, top_k)).astype(np.float32)
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    buf = torch.full((T * top_k, ld + 1), -7.0, dtype=z.dtype, device="cuda")
    dz, dw = mmq.moe_combine_grad(dy, z, plan, E, top_k, torch.from_numpy(w).cuda(), order=order, dz=buf[:, :N])
    got, dyh, zh = _host(buf), _host(dy), np.where(used[:, None], _host(z), 0.0)
    t, j = np.nonzero(row >= 0)
    want = np.full((T * top_k, ld + 1), -7.0)
    want[row[t, j], :N] = w[t, j, None].astype(np.float64) * dyh[t]
    off = np.abs(got - want)
    assert np.all(off[~used] == 0) and np.all(off[:, N:] == 0)
    step = U24 if dt == "f32" else U24 + U8 * (1 + U24)
    assert np.all(off <= np.abs(want) * step)
    terms = np.zeros((T, top_k, N))
    terms[t, j] = dyh[t] * zh[row[t, j]]
    # each lane sums its share of N, then lanes and waves join
    bound = np.abs(terms).sum(2) * (N + 10) * U24 * 1.01
    g = dw.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(g - terms.sum(2)) <= bound)
    assert np.all(g[row < 0] == 0)


def test_combine_grad_against_differences(env):
    """The gradients against central differences of the forward call's loss <y, c>, which is linear
    in z and in w, so that a difference of any step is the derivative up to rounding."""
    torch, mmq = env
    T, top_k, E, N = 6, 3, 4, 40
    ids = _ids(T, top_k, E, 0.2, 11)
    row = rowmodel.row_of(ids, E, "pair")
    g = torch.Generator().manual_seed(3)
    z, c = torch.randn((T * top_k, N), generator=g).cuda(), torch.randn((T, N), generator=g).cuda()
    w = torch.randn((T, top_k), generator=g).cuda()
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    dz, dw = mmq.moe_combine_grad(c, z, plan, E, top_k, w, dz=torch.zeros_like(z))
    loss = lambda zz, ww: (mmq.moe_combine(zz, plan, E, T, top_k, weights=ww).double() * c.double()).sum().item()  # noqa: E731
    scale = (w[:, :, None].abs() * z.view(T, top_k, N).abs() * c[:, None].abs()).sum().item()
    for t, j, n in ((0, 0, 0), (3, 1, 17), (5, 2, 39), (2, 2, 5)):
        p = t * top_k + j
        zp, zm, wp, wm = z.clone(), z.clone(), w.clone(), w.clone()
        zp[p, n] += 1
        zm[p, n] -= 1
        wp[t, j] += 1
        wm[t, j] -= 1
        # both losses are sums within 4 * 2^-24 of their terms' magnitudes (at most `scale` + the step's)
        tol = 2 * 4 * U24 * (scale + abs(float(c[t].abs().sum())) * 8)
        live = row[t, j] >= 0
        assert abs((loss(zp, w) - loss(zm, w)) / 2 - (dz[p, n].item() if live else 0.0)) <= tol
        assert abs((loss(z, wp) - loss(z, wm)) / 2 - dw[t, j].item()) <= tol


def test_row_calls_in_a_graph_and_on_a_stream(env):
    """Plan, gather, combination and gradients captured once and replayed with new ids and rows;
    each replay equals the eager calls, made on another stream, bit for bit."""
    torch, mmq = env
    T, top_k, E, N = 90, 4, 12, 333
    ids, x = torch.zeros((T, top_k), dtype=torch.int32, device="cuda"), torch.zeros((T, N), device="cuda")
    w, dy = torch.zeros((T, top_k), device="cuda"), torch.zeros((T, N), device="cuda")
    res = {}

    def path(stream=None):
        plan = mmq.group_rows(ids, E, stream=stream)
        rows = mmq.moe_gather(x, plan, E, top_k, stream=stream)
        y = mmq.moe_combine(rows, plan, E, T, top_k, weights=w, order="sorted", stream=stream)
        dz, dw = mmq.moe_combine_grad(dy, rows, plan, E, top_k, w, order="sorted", stream=stream)
        dx = mmq.moe_combine(dz, plan, E, T, top_k, order="sorted", stream=stream)
        return y, dw, dx
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        res["out"] = path()
    for rep in range(4):
        gen = torch.Generator().manual_seed(rep)
        ids.copy_(torch.from_numpy(_ids(T, top_k, E, 0.2, 20 + rep)))
        x.copy_(torch.randn((T, N), generator=gen))
        w.copy_(torch.randn((T, top_k), generator=gen))
        dy.copy_(torch.randn((T, N), generator=gen))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        other = torch.cuda.Stream()
        eager = path(other)                       # enqueued on `other`, whatever the current stream is
        other.synchronize()
        for a, b in zip(res["out"], eager):
            assert torch.equal(a, b), rep


def test_plan_must_fit(env):
    torch, mmq = env
    ids = torch.zeros((8, 2), dtype=torch.int32, device="cuda")
    plan = mmq.group_rows(ids, 4)
    with pytest.raises(ValueError, match="plan"):
        mmq.moe_gather(torch.zeros((4000, 8), device="cuda"), plan, 4, 2)
    with pytest.raises(ValueError, match="ids"):
        mmq.group_rows(ids.long(), 4)
    with pytest.raises(ValueError, match="ids"):
        mmq.group_rows(ids[:, :1], 4)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        mmq.moe_gather(torch.zeros((8, 8), device="cuda", dtype=torch.float16), plan, 4, 2)
    with pytest.raises(ValueError, match="weights"):
        mmq.moe_combine(torch.zeros((16, 8), device="cuda"), plan, 4, 8, 2, weights=torch.zeros((16, 1), device="cuda"))
    with pytest.raises(mmq.MMQError):
        mmq.group_rows(ids, 1)                     # top_k > E


def test_results_come_from_the_calls_own_stream(env):
    """A call on another stream gets no memory that work of the current stream may still be using."""
    torch, mmq = env
    other = torch.cuda.Stream()
    x = torch.zeros((64, 1000), device="cuda")
    ids = torch.zeros((64, 2), dtype=torch.int32, device="cuda")
    plan = mmq.group_rows(ids, 4)
    torch.cuda.synchronize()
    used = torch.empty((128, 1000), device="cuda")
    at = used.data_ptr()
    del used                                           # free for the current stream's next call alone
    rows = mmq.moe_gather(x, plan, 4, 2, stream=other)
    assert rows.data_ptr() != at
    other.synchronize()
    assert not bool(rows[:64].any())


def test_a_plan_of_another_batch_stays_inside_the_buffers(env):
    """The entries of a plan made for more tokens point past this batch's rows: the calls drop them."""
    torch, mmq = env
    T, big, top_k, E, N = 8, 1000, 2, 4, 64
    ids = torch.from_numpy(_ids(big, top_k, E, 0.0, 1)).cuda()
    plan = mmq.group_rows(ids, E)
    x, z = torch.ones((T, N), device="cuda"), torch.ones((T * top_k, N), device="cuda")
    frame = torch.full((T * top_k + 64, N), -7.0, device="cuda")
    mmq.moe_gather(x, plan, E, top_k, out=frame[:T * top_k])
    y = torch.full((T + 64, N), -7.0, device="cuda")
    mmq.moe_combine(z, plan, E, T, top_k, order="sorted", out=y[:T])
    torch.cuda.synchronize()
    assert bool((frame[T * top_k:] == -7.0).all()) and bool((y[T:] == -7.0).all())
    assert bool(((frame == 1.0) | (frame == -7.0)).all()) and bool(torch.isfinite(y).all())


@pytest.mark.parametrize("T,top_k,E,away", [
    (16384, 1, 64, 0.1), (16385, 1, 64, 0.1), (4096, 8, 64, 0.25), (9000, 2, 1023, 0.1),
    (9000, 2, 1024, 0.1), (262144, 3, 7, 0.0), (40000, 1, 4096, 0.5)])
def test_plans_of_one_and_of_two_launches(env, T, top_k, E, away):
    """Around the number of pairs, and of groups, where the sort changes its form."""
    test_plan_is_the_stable_sort(env, T, top_k, E, away)


@pytest.mark.parametrize("P", [1000, 16384, 50000])
def test_plan_of_runs(env, P):
    """Sorted ids: whole waves of one group, and everything in one."""
    torch, mmq = env
    print(f"[case] plan of runs P={P}", flush=True)
    for ids in (np.arange(P) * 5 // P, np.zeros(P), np.full(P, -1), np.arange(P) * 600 // P):
        ids = ids.astype(np.int32)
        plan = mmq.group_rows(torch.from_numpy(ids).cuda(), 600)
        for name, g, w in zip(("offs", "order", "pos", "units"), mmq.group_views(plan, 600, P), rowmodel.plan(ids, 600)):
            assert np.array_equal(g.cpu().numpy(), w), name


@pytest.mark.parametrize("order", ["pair", "sorted"])
@pytest.mark.parametrize("dims", [2, 3])
def test_gradient_rows_of_pairs_without_an_expert_are_zeros(env, order, dims):
    """Where the binding makes dz itself, it holds no earlier tensor's values: a row that the
    forward call does not read has a gradient of zeros."""
    torch, mmq = env
    T, top_k, E, N = 40, 3, 5, 70
    ids = _ids(T, top_k, E, 0.3, 12)
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    g = torch.Generator().manual_seed(1)
    z, dy = torch.randn((T * top_k, N), generator=g).cuda(), torch.randn((T, N), generator=g).cuda()
    w = torch.randn((T, top_k), generator=g).cuda()
    want, dw = mmq.moe_combine_grad(dy, z, plan, E, top_k, w, order=order, dz=torch.zeros_like(z))
    if dims == 3:
        z = z.view(T, top_k, N)
    for stream in (None, torch.cuda.Stream()):
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            used = [torch.full_like(z, float("nan")) for _ in range(4)]
        torch.cuda.synchronize()
        del used                                          # the next tensors of that size get this memory
        dz, dw2 = mmq.moe_combine_grad(dy, z, plan, E, top_k, w, order=order, stream=stream)
        torch.cuda.synchronize()
        assert dz.shape == z.shape and torch.equal(dz.view(-1, N), want) and torch.equal(dw2, dw)


@pytest.mark.parametrize("T,top_k,E,N,K,away", [(3, 2, 4, 96, 256, 0.0), (10, 8, 16, 130, 512, 0.2), (70, 3, 8, 97, 256, 0.2)])
def test_after_the_expert_products(env, T, top_k, E, N, K, away):
    """The run that the pair order is made for, as a layer makes it: quantise, the experts' products
    (mmq_gemm_id, of decode and of prefill sizes) into rows of pairs, the weighted sum of these rows
    as they come, [T, top_k, N], and its gradients; against the oracle's products and 64-bit sums."""
    torch, mmq = env
    import gen
    import oracle
    oracle.build()
    print(f"[case] gemm_id and combine T={T} top_k={top_k} E={E} N={N} K={K}", flush=True)
    raw = gen.moe_weights("q4_0", E, N, K, seed=2, cfg=143)
    xh = gen.act_f32(T, K, seed=3, cfg=143)
    ids = _ids(T, top_k, E, away, 13)
    pb = mmq.packed_bytes("q4_0", N, K)
    packed = torch.empty(E * pb, dtype=torch.uint8, device="cuda")
    for e in range(E):
        mmq.repack_weights("q4_0", torch.from_numpy(np.ascontiguousarray(raw[e])).cuda(), N, K, out=packed[e * pb:(e + 1) * pb])
    ids_d = torch.from_numpy(ids).cuda()
    act = mmq.quantize_act(torch.from_numpy(xh).cuda())
    z = torch.full((T, top_k, N), float("nan"), device="cuda")        # what the products leave unwritten
    mmq.gemm_id("q4_0", packed, E, act, ids_d, T, top_k, N, K, out=z)
    plan = mmq.group_rows(ids_d, E)
    g = torch.Generator().manual_seed(5)
    w = torch.randn((T, top_k), generator=g).softmax(1).cuda()
    dy = torch.randn((T, N), generator=g).cuda()
    y = mmq.moe_combine(z, plan, E, T, top_k, weights=w)
    dz, dw = mmq.moe_combine_grad(dy, z, plan, E, top_k, w)
    there = (ids >= 0)[:, :, None]
    rq, rs, _ = oracle.quantize_q8_1(xh)
    ref = np.where(there, oracle.moe_f64("q4_0", raw.reshape(E * N, -1), E, N, K, rq, rs, ids), 0.0)
    zh, wh = np.where(there, _host(z), 0.0), _host(w)[:, :, None]
    # softmax weights: the sum is off by no more than the products' own gate of their largest value
    assert np.max(np.abs(_host(y) - (wh * ref).sum(1))) <= 1e-3 * np.max(np.abs(ref))
    terms = wh * zh
    assert np.all(np.abs(_host(y) - terms.sum(1)) <= np.abs(terms).sum(1) * top_k * U24 * 1.01)
    want = np.where(there, wh * _host(dy)[:, None, :], 0.0)
    got = _host(dz)
    assert dz.shape == z.shape and np.all((np.abs(got - want) <= np.abs(want) * U24)[ids >= 0])
    terms = _host(dy)[:, None, :] * zh
    assert np.all(np.abs(_host(dw) - terms.sum(2)) <= np.abs(terms).sum(2) * (N + 10) * U24 * 1.01)
    assert not dw.cpu().numpy()[ids < 0].any()


@pytest.mark.parametrize("order", ["pair", "sorted"])
def test_gradient_rows_are_zeros_on_every_replay(env, order):
    """A captured call fills its dz again on each replay, where other ids leave other rows out."""
    torch, mmq = env
    T, top_k, E, N = 60, 3, 5, 130
    ids = torch.from_numpy(_ids(T, top_k, E, 0.3, 30)).cuda()
    z, dy, w = torch.randn((T, top_k, N), device="cuda"), torch.randn((T, N), device="cuda"), torch.randn((T, top_k), device="cuda")

    def path():
        return mmq.moe_combine_grad(dy, z, mmq.group_rows(ids, E), E, top_k, w, order=order)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dz, dw = path()
    for rep in range(4):
        ids.copy_(torch.from_numpy(_ids(T, top_k, E, 0.3, 31 + rep)))
        for t in (z, dy, w):
            t.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, dww = mmq.moe_combine_grad(dy, z, mmq.group_rows(ids, E), E, top_k, w, order=order, dz=torch.zeros_like(z))
        assert torch.equal(dz, want) and torch.equal(dw, dww), rep
