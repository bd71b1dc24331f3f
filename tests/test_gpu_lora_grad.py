"""The adapters' gradients from 8-bit activations on the GPU, through the public binding, against
64-bit sums and against differences of the forward call.

Tolerances, as for the forward call: products of operands are exact in f32 (dy and v, and u with
the block scale, as three bf16 terms each; the term pairs left out are below 2^-23 of the
product; u times a block scale is rounded once, 2^-24), each of a sum's n additions is off by at
most 2^-23 of the running sum. u is a sum over N of products of up to five term pairs; dB one
over the adapter's rows (six pairs); dA one over the rows of products with u (three pairs); dx
adds R products (five pairs) to its base."""
import numpy as np
import pytest

import rowmodel
from test_gpu_lora import activations, adapters, host, row_ids

pytestmark = pytest.mark.gpu

U23, U24 = 2.0 ** -23, 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    import block_quantized_int8_amd as mmq
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mmq.lib()
    return torch, mmq


def problem(torch, mmq, act, kind, M, N, K, R, E, how, seed=1):
    ids = row_ids(M, E, how, seed)
    buf, x = activations(mmq, act, M, K, seed + 1)
    A, B, scale = adapters(torch, kind, E, R, K, N, seed + 2)
    io = torch.float32 if act == "q8_1" else torch.bfloat16
    g = torch.Generator().manual_seed(seed + 3)
    dy = (torch.randn((M, N), generator=g) * 0.1).to(io)
    v = torch.from_numpy(rowmodel.lora(x, host(A), host(B), host(scale), ids, np.zeros((M, N)))[1]).float()
    dxb = torch.randn((M, K), generator=g)
    return ids, buf, x, A, B, scale, dy, v, dxb


CASES = [
    ("q8_1", "bf16", 1, 1, 32, 8, 1, "one"), ("i8_token", "f16", 1, 3, 32, 8, 2, "one"),
    ("q8_1", "f16", 2, 4099, 96, 16, 3, "mixed"), ("q8_1", "bf16", 31, 257, 96, 16, 3, "mixed"),
    ("i8_token", "bf16", 33, 255, 64, 24, 2, "mixed"), ("q8_1", "f16", 64, 64, 416, 32, 5, "mixed"),
    ("q8_1", "bf16", 65, 1003, 1024, 40, 1, "one"), ("i8_token", "f16", 129, 129, 320, 64, 4, "runs"),
    ("q8_1", "bf16", 150, 512, 288, 64, 64, "mixed"), ("q8_1", "f16", 200, 130, 1056, 72, 2, "runs"),
    ("i8_token", "bf16", 130, 70, 544, 128, 3, "runs"), ("q8_1", "bf16", 200, 301, 512, 256, 2, "runs"),
    ("q8_1", "f16", 333, 99, 800, 8, 70, "mixed"), ("i8_token", "f16", 301, 777, 96, 16, 1, "one"),
    ("q8_1", "bf16", 40, 50, 64, 16, 3, "none"), ("q8_1", "bf16", 1000, 260, 128, 48, 4, "runs"),
    ("i8_token", "bf16", 100, 33, 4128, 8, 2, "runs"), ("q8_1", "bf16", 41, 10342, 96, 64, 4, "mixed"),
    ("i8_token", "f16", 20, 4129, 64, 24, 2, "mixed"), ("q8_1", "f16", 70, 8193, 32, 136, 1, "one"), ("q8_1", "bf16", 90, 65, 64, 8, 4096, "mixed"),
]


@pytest.mark.parametrize("act,kind,M,N,K,R,E,how", CASES)
def test_gradients(env, act, kind, M, N, K, R, E, how):
    torch, mmq = env
    print(f"[case] lora_grad {act} {kind} M={M} N={N} K={K} R={R} E={E} {how}", flush=True)
    ids, buf, x, A, B, scale, dy, v, dxb = problem(torch, mmq, act, kind, M, N, K, R, E, how)
    dev = [t.cuda() for t in (torch.from_numpy(buf), A, B, scale)]
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    dyf = torch.full((M, N + 1), float("nan"), dtype=dy.dtype, device="cuda")     # columns past N are not read
    dyf[:, :N] = dy.cuda()
    none = torch.from_numpy((ids < 0) | (ids >= E))
    dyf[none.cuda()] = float("nan")                                              # nor rows without an adapter
    dxf = torch.full((M, K + 3), -7.0, device="cuda")
    dxf[:, :K] = dxb.cuda()
    dA = torch.full((E, R, K), float("nan"), device="cuda")
    dB = torch.full((E, N, R), float("nan"), device="cuda")
    mmq.lora_grad(*dev, plan, v.cuda(), dyf[:, :N], atype=act, dx_base=dxf[:, :K], dx=dxf[:, :K], dA=dA, dB=dB)
    want, mag = rowmodel.lora_grad(x, host(A), host(B), host(scale), ids, host(v), host(dy), host(dxb))
    rows = max(1, int(np.bincount(ids[~none.numpy()], minlength=1).max()) if (~none).any() else 1)
    nu = 5 * N + 8                                   # additions behind a value of u
    for name, got, w, m, n in (("dB", dB, want[2], mag[2], 6 * rows + 8), ("dA", dA, want[1], mag[1], nu + 3 * rows + 10),
                               ("dx", dxf[:, :K], want[0], mag[0], nu + 5 * R + 8)):
        assert np.all(np.abs(host(got) - w) <= n * U23 * m * 1.01), name
        if np.linalg.norm(w):                        # and, in the mean, as near as f32 sums are
            assert np.linalg.norm(host(got) - w) <= 1e-6 * np.linalg.norm(w), name
    assert np.all(host(dxf)[:, K:] == -7.0)
    assert torch.equal(dxf[:, :K].cpu()[none], dxb[none])
    for e in range(min(E, 8)):
        if not np.any(ids == e):
            assert not dA[e].any() and not dB[e].any()
    # out of place: the same bits; without a base and without dx too
    dx2, dA2, dB2 = mmq.lora_grad(*dev, plan, v.cuda(), dy.cuda(), atype=act, dx_base=dxb.cuda())
    assert torch.equal(dx2, dxf[:, :K]) and torch.equal(dA2, dA) and torch.equal(dB2, dB)
    dx0, dA0, dB0 = mmq.lora_grad(*dev, plan, v.cuda(), dy.cuda(), atype=act)
    assert np.all(np.abs(host(dx0) - (want[0] - host(dxb))) <= (nu + 5 * R + 8) * U23 * mag[0] * 1.01)
    assert not dx0.cpu()[none].any() and torch.equal(dA0, dA)
    nothing, dA0, dB0 = mmq.lora_grad(*dev, plan, v.cuda(), dy.cuda(), atype=act, want_dx=False)
    assert nothing is None and torch.equal(dA0, dA) and torch.equal(dB0, dB)


@pytest.mark.parametrize("act", ["q8_1", "i8_token"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,R,E", [(1, 70, 64, 8, 1), (70, 100, 96, 16, 3), (150, 130, 64, 40, 2)])
def test_gradients_exact_on_integers(env, act, kind, M, N, K, R, E):
    """Integers whose sums stay below 2^24 but need more bits than two bf16 terms hold: nothing
    rounds, so the gradients have to be equal."""
    torch, mmq = env
    print(f"[case] lora_grad integers {act} {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    r = np.random.default_rng([M, N, K, R])
    ids = row_ids(M, E, "mixed", 5)
    q = (r.integers(-2, 3, (M, K)) * (r.random((M, K)) < 0.2)).astype(np.int8)
    s = np.ones((M, K // 32) if act == "q8_1" else M, np.float32)
    buf = mmq.act_q8_1_pack_host(q, s) if act == "q8_1" else mmq.act_i8_pack_host(q, s)
    top, big = (255, 2047) if kind == "bf16" else (2047, 255)
    A = (r.integers(-2, 3, (E, R, K)) * (r.random((E, R, K)) < 0.2)).astype(np.float32)
    B = (r.integers(-top, top + 1, (E, N, R)) * (r.random((E, N, R)) < 2 / N)).astype(np.float32)
    if act == "i8_token":
        big = 127                                       # what bf16 gradients hold
    dy = (r.integers(-big, big + 1, (M, N)) * (r.random((M, N)) < 0.1)).astype(np.float32)
    if act == "q8_1":                                   # gradients of 18 bits where B is 0
        B[:, ::7] = 0
        dy[:, ::7] = r.integers(-(1 << 17), 1 << 17, dy[:, ::7].shape) * (r.random(dy[:, ::7].shape) < 0.1)
    v = r.integers(-3, 4, (M, R)).astype(np.float32)
    dxb = r.integers(-99, 100, (M, K)).astype(np.float32)
    scale = np.ones(E, np.float32)
    want, mag = rowmodel.lora_grad(q.astype(np.float64), A, B, scale, ids, v, dy, dxb)
    assert max(m.max() for m in mag) < 2 ** 24
    dt, io = (torch.bfloat16 if kind == "bf16" else torch.float16), (torch.float32 if act == "q8_1" else torch.bfloat16)
    got = mmq.lora_grad(torch.from_numpy(buf).cuda(), torch.from_numpy(A).to(dt).cuda(), torch.from_numpy(B).to(dt).cuda(),
                        torch.from_numpy(scale).cuda(), mmq.group_rows(torch.from_numpy(ids).cuda(), E),
                        torch.from_numpy(v).cuda(), torch.from_numpy(dy).to(io).cuda(), atype=act,
                        dx_base=torch.from_numpy(dxb).cuda())
    for name, g, w in zip(("dx", "dA", "dB"), got, want):
        assert np.array_equal(host(g), w), name


def test_against_differences_of_the_forward_call(env):
    """loss = <out, c> is linear in A and in B, so a central difference of any step is the
    derivative up to the rounding of the two forward calls (each within (K + 5 R + 16) 2^-23 of
    its terms' magnitudes)."""
    torch, mmq = env
    M, N, K, R, E = 50, 70, 96, 16, 3
    ids, buf, x, A, B, scale, c, _, _ = problem(torch, mmq, "q8_1", "bf16", M, N, K, R, E, "runs", seed=9)
    act, scale_d, c_d = torch.from_numpy(buf).cuda(), scale.cuda(), c.cuda()
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    forward = lambda a, b: mmq.lora(act, a, b, scale_d, plan, M)     # noqa: E731
    loss = lambda a, b: (forward(a, b)[0].double() * c_d.double()).sum().item()      # noqa: E731
    A, B = A.cuda(), B.cuda()
    v = forward(A, B)[1]
    _, dA, dB = mmq.lora_grad(act, A, B, scale_d, plan, v, c_d)
    mag = rowmodel.lora(x, np.abs(host(A)) + 0.5, np.abs(host(B)) + 0.5, host(scale), ids, np.zeros((M, N)))[2]
    tol = 2 * (K + 5 * R + 16) * U23 * float((mag * np.abs(host(c))).sum())
    for e, i, j in ((0, 0, 0), (1, 7, 33), (2, 15, 69), (1, 12, 5)):
        ap, am, bp, bm = A.clone(), A.clone(), B.clone(), B.clone()
        ap[e, i, j] += 0.5
        am[e, i, j] -= 0.5
        bp[e, j, i] += 0.5
        bm[e, j, i] -= 0.5
        step_a, step_b = (ap - am)[e, i, j].item(), (bp - bm)[e, j, i].item()     # as the bf16 values moved
        assert abs((loss(ap, B) - loss(am, B)) / step_a - dA[e, i, j].item()) <= tol / 0.5
        assert abs((loss(A, bp) - loss(A, bm)) / step_b - dB[e, j, i].item()) <= tol / 0.5
    # and for the activations: their step goes through the formula out = s B A x^ itself
    dx, _, _ = mmq.lora_grad(act, A, B, scale_d, plan, v, c_d)
    full = np.zeros((M, K))
    for e in range(E):
        at = np.nonzero(ids == e)[0]
        full[at] = host(scale)[e] * (host(c)[at] @ host(B)[e] @ host(A)[e])
    assert np.linalg.norm(host(dx) - full) <= 1e-6 * np.linalg.norm(full)


def test_a_training_step(env):
    """Forward and backward of one projection with its adapters, as a training step runs them:
    quantise once, project, add the adapters; their gradients from the same act buffer. An SGD step
    along the gradients changes the loss by what the gradients say."""
    torch, mmq = env
    import gen
    M, N, K, R, E = 96, 160, 256, 8, 2
    raw = gen.weights("q8_0", N, K, seed=5, cfg=142)
    packed = mmq.repack_weights("q8_0", torch.from_numpy(raw).cuda(), N, K)
    x = torch.from_numpy(gen.act_f32(M, K, seed=6, cfg=142)).cuda()
    ids = torch.from_numpy(row_ids(M, E, "runs", 3)).cuda()
    A, B, scale = (t.cuda() for t in adapters(torch, "bf16", E, R, K, N, 4))
    target = torch.randn((M, N), generator=torch.Generator().manual_seed(1)).cuda()
    plan = mmq.group_rows(ids, E)

    def forward(a, b):
        act = mmq.quantize_act(x)
        out = mmq.gemm("q8_0", packed, act, M, N, K)
        out, v = mmq.lora(act, a, b, scale, plan, M, base=out, out=out)
        return act, out, v
    act, out, v = forward(A, B)
    dy = (out - target) * (2.0 / (M * N))
    _, dA, dB = mmq.lora_grad(act, A, B, scale, plan, v, dy, want_dx=False)
    A64, B64 = A.double().requires_grad_(), B.double().requires_grad_()
    xh = torch.from_numpy(rowmodel.act_values("q8_1", *mmq.act_to_host(act.cpu().numpy(), M, K)[:2])).cuda()
    proj = mmq.gemm("q8_0", packed, act, M, N, K).double()
    pick = ids.long().clamp(min=0)
    ok = (ids >= 0).double()[:, None]
    vv = (xh[:, None, :] * A64[pick]).sum(2) * ok
    loss = ((proj + scale.double()[pick][:, None] * (vv[:, None, :] * B64[pick]).sum(2) - target.double()) ** 2).mean()
    loss.backward()
    # dy carries the f32 rounding of `out` and of the difference: 2^-23 of their magnitudes each
    for got, want in ((dA, A64.grad), (dB, B64.grad)):
        assert ((got.double() - want).norm() / want.norm()).item() <= 1e-5


def test_graph_and_streams(env):
    torch, mmq = env
    M, N, K, R, E = 77, 300, 256, 32, 6
    A, B, scale = (t.cuda() for t in adapters(torch, "f16", E, R, K, N, 8))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    act = torch.zeros(mmq.act_bytes("i8_token", M, K), dtype=torch.uint8, device="cuda")
    v, dxb = torch.zeros((M, R), device="cuda"), torch.zeros((M, K), device="cuda")
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    got = {}

    def path(stream=None):
        plan = mmq.group_rows(ids, E, stream=stream)
        return mmq.lora_grad(act, A, B, scale, plan, v, dy, atype="i8_token", dx_base=dxb, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got["out"] = path()
    for rep in range(4):
        act.copy_(torch.from_numpy(activations(mmq, "i8_token", M, K, 40 + rep)[0]))
        ids.copy_(torch.from_numpy(row_ids(M, E, ["mixed", "runs", "one", "none"][rep], rep)))
        for t in (v, dxb, dy):
            t.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        every = [path(s) for s in (s1, s2, s1, s2)]
        torch.cuda.synchronize()
        for res in every:
            for a, b in zip(res, got["out"]):
                assert torch.equal(a, b), rep


@pytest.mark.parametrize("act", ["q8_1", "i8_token"])
@pytest.mark.parametrize("M,N,K,R,E", [(1, 70, 64, 8, 1), (70, 100, 96, 16, 3), (150, 130, 64, 40, 2), (300, 6500, 64, 72, 2)])
def test_gradients_exact_far_from_one(env, act, M, N, K, R, E):
    """Integers times powers of two: f16 adapters below the smallest normal value, gradients near
    2^-60 (what a loss's mean leaves); nothing rounds, so the gradients have to be equal."""
    torch, mmq = env
    print(f"[case] lora_grad scaled {act} M={M} N={N} K={K} R={R} E={E}", flush=True)
    r = np.random.default_rng([M, N, K, R])
    ids = row_ids(M, E, "mixed", 5)
    q = (r.integers(-2, 3, (M, K)) * (r.random((M, K)) < 0.2)).astype(np.int8)
    s = np.ones((M, K // 32) if act == "q8_1" else M, np.float32)
    buf = mmq.act_q8_1_pack_host(q, s) if act == "q8_1" else mmq.act_i8_pack_host(q, s)
    A = (r.integers(-2, 3, (E, R, K)) * (r.random((E, R, K)) < 0.2) * 2.0 ** -24).astype(np.float32)
    B = (r.integers(-1023, 1024, (E, N, R)) * (r.random((E, N, R)) < 2 / N) * 2.0 ** -24).astype(np.float32)
    dy = (r.integers(-127, 128, (M, N)) * (r.random((M, N)) < 0.1) * 2.0 ** -60).astype(np.float32)
    v = (r.integers(-3, 4, (M, R)) * 2.0 ** -30).astype(np.float32)
    scale = np.ones(E, np.float32)
    want, mag = rowmodel.lora_grad(q.astype(np.float64), A, B, scale, ids, v, dy, np.zeros((M, K)))
    for m, unit in zip(mag, (-108, -84, -90)):                   # dx, dA, dB in units of their products
        assert m.max() < 2.0 ** (24 + unit)
    io = torch.float32 if act == "q8_1" else torch.bfloat16
    got = mmq.lora_grad(torch.from_numpy(buf).cuda(), torch.from_numpy(A).half().cuda(), torch.from_numpy(B).half().cuda(),
                        torch.from_numpy(scale).cuda(), mmq.group_rows(torch.from_numpy(ids).cuda(), E),
                        torch.from_numpy(v).cuda(), torch.from_numpy(dy).to(io).cuda(), atype=act)
    for name, g, w in zip(("dx", "dA", "dB"), got, want):
        assert np.array_equal(host(g), w), name


@pytest.mark.parametrize("act,kind,M,N,K,R,E", [
    ("q8_1", "f16", 5, 70, 64, 16, 3), ("q8_1", "bf16", 400, 300, 128, 72, 3), ("i8_token", "bf16", 150, 131, 96, 64, 2),
    ("i8_token", "f16", 90, 6500, 64, 32, 4)])
def test_what_is_not_finite_stays_with_its_adapter(env, act, kind, M, N, K, R, E):
    """A row whose dy is not finite in one column, of an adapter: other rows' dx, other adapters' dA
    and dB and the adapter's dB of other columns stay bit for bit, whatever the workspace held."""
    torch, mmq = env
    print(f"[case] lora_grad not finite {act} {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    ids, buf, x, A, B, scale, dy, v, dxb = problem(torch, mmq, act, kind, M, N, K, R, E, "runs", seed=5)
    at, e, n = M // 2, E - 1, N - 2
    ids[at] = e
    v[at] = 1.0
    dev = [t.cuda() for t in (torch.from_numpy(buf), A, B, scale)]
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    need = mmq.lora_grad_workspace_bytes(E, M, N, K, R)

    def run(g, fill):
        return mmq.lora_grad(*dev, plan, v.cuda(), g.cuda(), atype=act, dx_base=dxb.cuda(),
                             workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
    clean = run(dy, 0)
    assert all(bool(t.isfinite().all()) for t in clean)
    others = [i for i in range(M) if i != at]
    for value in (float("nan"), float("inf"), float("-inf")):
        bad = dy.clone()
        bad[at, n] = value
        dx, dA, dB = run(bad, 255)
        assert torch.equal(dx[others], clean[0][others]) and not bool(dx[at].isfinite().any())
        assert torch.equal(dA[:e], clean[1][:e]) and torch.equal(dB[:e], clean[2][:e])
        assert not bool(dA[e].isfinite().any()) and not bool(dB[e, n].isfinite().any())
        cols = [i for i in range(N) if i != n]
        assert torch.equal(dB[e, cols], clean[2][e, cols])


@pytest.mark.parametrize("act,kind,M,N,K,R,E,big", [
    ("q8_1", "bf16", 900, 70, 96, 16, 200, (150,)), ("i8_token", "f16", 700, 300, 64, 40, 129, (0, 63, 64, 128)),
    ("q8_1", "f16", 400, 65, 64, 8, 2, (1,)), ("q8_1", "bf16", 1100, 33, 11008, 8, 4, (0, 1, 2, 3)),
    ("i8_token", "bf16", 1100, 16500, 32, 8, 4, (0, 1, 2, 3)), ("q8_1", "bf16", 640, 500, 160, 72, 6, (2, 5))])
def test_adapters_of_many_and_of_few_rows(env, act, kind, M, N, K, R, E, big):
    """Nearly all rows with a few adapters (some of them past the 64th), the rest with a few rows or
    none; more blocks of output than workgroups that share them."""
    torch, mmq = env
    print(f"[case] lora_grad many {act} {kind} M={M} N={N} K={K} R={R} E={E} {big}", flush=True)
    _, buf, x, A, B, scale, dy, v, dxb = problem(torch, mmq, act, kind, M, N, K, R, E, "none", seed=6)
    r = np.random.default_rng([M, E])
    ids = np.asarray(big, np.int32)[np.arange(M) % len(big)]
    few = r.random(M) < 0.03
    ids[few] = r.integers(-1, E, int(few.sum()))
    v = torch.randn((M, R), generator=torch.Generator().manual_seed(2))
    got = mmq.lora_grad(*(t.cuda() for t in (torch.from_numpy(buf), A, B, scale)),
                        mmq.group_rows(torch.from_numpy(ids).cuda(), E), v.cuda(), dy.cuda(), atype=act, dx_base=dxb.cuda())
    want, mag = rowmodel.lora_grad(x, host(A), host(B), host(scale), ids, host(v), host(dy), host(dxb))
    rows, nu = int(np.bincount(ids[ids >= 0]).max()), 5 * N + 8
    for name, g, w, m, n in zip(("dx", "dA", "dB"), got, want, mag, (nu + 5 * R + 8, nu + 3 * rows + 10, 6 * rows + 8)):
        assert np.all(np.abs(host(g) - w) <= n * U23 * m * 1.01), name
        assert np.linalg.norm(host(g) - w) <= 1e-6 * np.linalg.norm(w), name


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,R,E", [(5, 70, 64, 8, 5), (300, 131, 96, 40, 2), (20, 6500, 64, 72, 2)])
def test_a_single_product_keeps_f32(env, kind, M, N, K, R, E):
    """One row of each adapter has a gradient; its dy and v have 24 bits, a rank one weight, the
    scale is a power of two. dB is one product of f32 values and u one of an f32 value with a weight:
    all pairs of terms are added but one below 2^-30 of the product, the small ones first, so
    that only additions round. The last is off by at most 2^-23 of the result, those before it by
    2^-23 of partial sums that are below 2^-6, 2^-7 and far less of it; together with the pair
    below (1 + 2^-4) 2^-23. dA is u itself (x^ = 1), dx one product of u."""
    torch, mmq = env
    print(f"[case] lora_grad one product {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    r = np.random.default_rng([M, N, K, R])
    wbits = 11 if kind == "f16" else 8
    ids = (np.arange(M) % E).astype(np.int32)
    hot = np.arange(M - E, M)                             # the last rows: one of each adapter
    e_of = ids[hot]
    dy, v = np.zeros((M, N), np.float32), np.zeros((M, R), np.float32)
    dy[hot] = rowmodel.full_significands(r, (E, N), 24) * 2.0 ** -23
    v[hot] = rowmodel.full_significands(r, (E, R), 24) * 2.0 ** -23
    A, B = np.zeros((E, R, K), np.float32), np.zeros((E, N, R), np.float32)
    n_of, r_of = r.integers(0, N, R), r.integers(0, R, K)
    B[:, n_of, np.arange(R)] = rowmodel.full_significands(r, (E, R), wbits) * 2.0 ** (1 - wbits)
    A[:, r_of, np.arange(K)] = rowmodel.full_significands(r, (E, K), wbits) * 2.0 ** (1 - wbits)
    scale = (2.0 ** (np.arange(E) % 3 - 1)).astype(np.float32)
    buf = mmq.act_q8_1_pack_host(np.ones((M, K), np.int8), np.ones((M, K // 32), np.float32))
    dt = torch.float16 if kind == "f16" else torch.bfloat16
    dx, dA, dB = mmq.lora_grad(torch.from_numpy(buf).cuda(), torch.from_numpy(A).to(dt).cuda(),
                               torch.from_numpy(B).to(dt).cuda(), torch.from_numpy(scale).cuda(),
                               mmq.group_rows(torch.from_numpy(ids).cuda(), E), torch.from_numpy(v).cuda(),
                               torch.from_numpy(dy).cuda())
    s, one = scale[e_of].astype(np.float64), (1 + 2.0 ** -4) * U23
    want = s[:, None, None] * dy[hot].astype(np.float64)[:, :, None] * v[hot][:, None, :]
    assert np.all(np.abs(host(dB)[e_of] - want) <= one * want)
    u = s[:, None] * dy[hot].astype(np.float64)[:, n_of] * B[e_of][:, n_of, np.arange(R)]
    got = host(dA)[e_of]
    assert np.all(np.abs(got - u[:, :, None]) <= one * u[:, :, None])
    want = u[:, r_of] * A[e_of][:, r_of, np.arange(K)]
    assert np.all(np.abs(host(dx)[hot] - want) <= one * (2 + one) * want)


def test_no_dx_where_none_is_wanted(env):
    """want_dx=False returns None and writes no dx, given or not."""
    torch, mmq = env
    ids, buf, _, A, B, scale, dy, v, dxb = problem(torch, mmq, "q8_1", "bf16", 40, 70, 64, 16, 3, "runs")
    args = [t.cuda() for t in (torch.from_numpy(buf), A, B, scale)] + [mmq.group_rows(torch.from_numpy(ids).cuda(), 3)]
    args += [v.cuda(), dy.cuda()]
    _, dA, dB = mmq.lora_grad(*args)
    dx = torch.full((40, 64), -7.0, device="cuda")
    got = mmq.lora_grad(*args, dx=dx, dx_base=dxb.cuda(), want_dx=False)
    assert got[0] is None and torch.equal(got[1], dA) and torch.equal(got[2], dB)
    assert bool((dx == -7.0).all())


def test_dx_of_rows_without_an_adapter_is_its_base_bit_for_bit(env):
    torch, mmq = env
    ids, buf, _, A, B, scale, dy, v, dxb = problem(torch, mmq, "q8_1", "bf16", 90, 70, 96, 16, 3, "mixed")
    away = torch.from_numpy((ids < 0) | (ids >= 3))
    for i, value in enumerate((-0.0, 0.0, 1e-40, float("inf"), -float("inf"))):
        dxb[:, i::11] = value
    dx, _, _ = mmq.lora_grad(*(t.cuda() for t in (torch.from_numpy(buf), A, B, scale)),
                             mmq.group_rows(torch.from_numpy(ids).cuda(), 3), v.cuda(), dy.cuda(), dx_base=dxb.cuda())
    assert bool(away.any()) and torch.equal(dx.cpu()[away].view(torch.int32), dxb[away].view(torch.int32))
