"""Low-rank adapters beside a shared projection on the GPU, through the public binding, against
64-bit sums.

Tolerances. Every product of operands is exact in f32; a sum of n terms made by the matrix core
and by fused multiply-adds, each addition cut off or rounded (off by at most 2^-23 of the running
sum), is off by at most n * 2^-23 * sum |terms|. v is such a sum over K; out adds the R products
of v (three or five terms each, the pairs left out below 2^-23 of the product) to that error, and
is rounded once to its type (2^-24 or 2^-8). On inputs whose every partial sum is an integer below
2^24 nothing rounds, and the results have to be equal."""
import numpy as np
import pytest

import gen
import rowmodel

pytestmark = pytest.mark.gpu

U23, U24, U8 = 2.0 ** -23, 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def env():
    import torch
    import block_quantized_int8_amd as mmq
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mmq.lib()
    return torch, mmq


def row_ids(M, E, how, seed):
    r = np.random.default_rng([seed, M, E])
    if how == "none":
        return np.full(M, -1, np.int32)
    if how == "one":                              # one request
        return np.full(M, E - 1, np.int32)
    if how == "mixed":
        ids = r.integers(0, E, M).astype(np.int32)
        if M > 1:
            ids[r.random(M) < 0.15] = r.choice([-1, E, 1 << 30, -(1 << 31)])
        return ids
    cuts = np.sort(r.integers(0, M, E))           # runs of requests, some empty; a run without adapter
    ids = np.searchsorted(cuts, np.arange(M), side="right").astype(np.int32)
    return np.where(ids == E, -1, ids).astype(np.int32)


def adapters(torch, kind, E, R, K, N, seed):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    A = (torch.randn((E, R, K), generator=g) * K ** -0.5).to(dt)
    B = (torch.randn((E, N, R), generator=g) * 0.1).to(dt)
    scale = 0.25 + torch.rand((E,), generator=g)
    return A, B, scale


def activations(mmq, kind, M, K, seed):
    """An act buffer (host bytes) and the 64-bit values it stands for."""
    x = gen.act_f32(M, K, seed=seed, cfg=140, outlier_rate=1e-2)
    amax = np.abs(x.reshape(M, K // 32, 32)).max(2) if kind == "q8_1" else np.abs(x).max(1)
    s = (amax / np.float32(127)).astype(np.float32)
    per = np.repeat(s, 32, axis=1) if kind == "q8_1" else s[:, None]
    q = np.clip(np.rint(x / per), -128, 127).astype(np.int8)
    if kind == "q8_1":
        s = s.astype(np.float16).astype(np.float32)
        return mmq.act_q8_1_pack_host(q, s), rowmodel.act_values(kind, q, s)
    return mmq.act_i8_pack_host(q, s), rowmodel.act_values(kind, q, s)


def host(t):
    return t.float().cpu().numpy().astype(np.float64)


CASES = [
    ("q8_1", "bf16", 1, 1, 32, 8, 1, "one"), ("i8_token", "f16", 1, 3, 32, 8, 1, "one"),
    ("q8_1", "f16", 1, 4096, 4096, 16, 8, "one"), ("q8_1", "bf16", 2, 257, 96, 16, 3, "mixed"),
    ("i8_token", "bf16", 5, 255, 64, 24, 2, "mixed"), ("q8_1", "f16", 16, 64, 416, 32, 5, "mixed"),
    ("q8_1", "bf16", 17, 1003, 1024, 40, 1, "one"), ("i8_token", "f16", 63, 129, 320, 64, 4, "runs"),
    ("q8_1", "bf16", 64, 512, 288, 64, 64, "mixed"), ("q8_1", "f16", 65, 130, 1056, 72, 2, "runs"),
    ("i8_token", "bf16", 130, 70, 544, 128, 3, "runs"), ("q8_1", "bf16", 200, 301, 512, 256, 2, "runs"),
    ("q8_1", "f16", 333, 99, 800, 8, 70, "mixed"), ("i8_token", "f16", 301, 777, 96, 16, 1, "one"),
    ("q8_1", "bf16", 40, 50, 64, 16, 3, "none"), ("q8_1", "bf16", 700, 260, 128, 48, 4, "runs"),
    ("i8_token", "bf16", 100, 33, 11008, 8, 2, "runs"), ("q8_1", "bf16", 90, 65, 64, 8, 4096, "mixed"),
]


@pytest.mark.parametrize("act,kind,M,N,K,R,E,how", CASES)
def test_forward(env, act, kind, M, N, K, R, E, how):
    torch, mmq = env
    print(f"[case] lora {act} {kind} M={M} N={N} K={K} R={R} E={E} {how}", flush=True)
    ids = row_ids(M, E, how, 1)
    buf, x = activations(mmq, act, M, K, 2)
    A, B, scale = adapters(torch, kind, E, R, K, N, 3)
    io = torch.float32 if act == "q8_1" else torch.bfloat16
    frame = torch.full((M, N + 3), -7.0, dtype=io, device="cuda")
    frame[:, :N] = torch.randn((M, N), generator=torch.Generator().manual_seed(4)).to(io).cuda()
    base = frame[:, :N].clone()
    dev = [t.cuda() for t in (torch.from_numpy(buf), A, B, scale)]
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    v = torch.full((M, R), float("nan"), device="cuda")
    out, v = mmq.lora(*dev, plan, M, atype=act, base=frame[:, :N], out=frame[:, :N], v=v)     # in place
    want, wv, mag, mag_v = rowmodel.lora(x, host(A), host(B), host(scale), ids, host(base))
    got, gv = host(frame), host(v)
    assert np.all(got[:, N:] == -7.0)
    assert np.all(np.abs(gv - wv) <= (K + 8) * U23 * mag_v * 1.01)
    tol = (K + 8 + 5 * R + 8) * U23 * mag * 1.01
    tol += (np.abs(want) + tol) * (U24 if act == "q8_1" else U8)
    assert np.all(np.abs(got[:, :N] - want) <= tol)
    none = (ids < 0) | (ids >= E)
    assert np.all(gv[none] == 0)
    assert torch.equal(frame[:, :N].cpu()[torch.from_numpy(none)], base.cpu()[torch.from_numpy(none)])
    # much nearer than the bounds where the terms have both signs: as near as f32 sums are
    if act == "q8_1" and how != "none":
        assert np.linalg.norm(gv - wv) <= 1e-6 * np.linalg.norm(wv)
    # out of place, twice: the same bits
    for _ in range(2):
        out2, v2 = mmq.lora(*dev, plan, M, atype=act, base=base)
        assert torch.equal(out2, frame[:, :N]) and torch.equal(v2, v)
    # no base: zeros
    out0, _ = mmq.lora(*dev, plan, M, atype=act)
    want0 = want - host(base)
    tol0 = (K + 8 + 5 * R + 8) * U23 * mag * 1.01
    tol0 += (np.abs(want0) + tol0) * (U24 if act == "q8_1" else U8)
    assert np.all(np.abs(host(out0) - want0) <= tol0)
    assert np.all(host(out0)[none] == 0)


def integer_case(mmq, act, kind, M, N, K, R, E, seed):
    """Inputs of small integers (times powers of two) whose sums need up to 24 bits."""
    r = np.random.default_rng(seed)
    q = r.integers(-127, 128, (M, K)).astype(np.int8)
    if act == "q8_1":
        s = (2.0 ** r.integers(0, 2, (M, K // 32))).astype(np.float32)
        buf = mmq.act_q8_1_pack_host(q, s)
    else:
        s = (2.0 ** r.integers(0, 2, M)).astype(np.float32)
        buf = mmq.act_i8_pack_host(q, s)
    top = 255 if kind == "bf16" else 2047                     # 8 and 11 significand bits
    A = r.integers(-top, top + 1, (E, R, K)) * (r.random((E, R, K)) < (24 if kind == "bf16" else 4) / max(K, 64))
    B = r.integers(-2, 3, (E, N, R)) * (r.random((E, N, R)) < 2 / R)
    return buf, rowmodel.act_values(act, q, s), A.astype(np.float32), B.astype(np.float32)


@pytest.mark.parametrize("act", ["q8_1", "i8_token"])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,R,E", [(1, 70, 64, 8, 1), (33, 100, 256, 16, 3), (150, 300, 512, 64, 2), (70, 65, 96, 136, 2)])
def test_forward_exact_on_integers(env, act, kind, M, N, K, R, E):
    torch, mmq = env
    print(f"[case] lora integers {act} {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    buf, x, A, B = integer_case(mmq, act, kind, M, N, K, R, E, [M, N, K])
    ids = row_ids(M, E, "mixed", 5)
    scale = 2.0 ** (np.arange(E) % 2) / 2
    base = np.random.default_rng(6).integers(-64, 65, (M, N)).astype(np.float32)
    want, wv, mag, mag_v = rowmodel.lora(x, A, B, scale, ids, base)
    assert mag_v.max() < 2 ** 24 and (2 * mag).max() < 2 ** 25      # halves of integers below 2^24
    if mag_v.max() > 2 ** 17:
        assert np.any(np.abs(wv) > 2 ** 16)                         # more bits than two terms hold
    dt, io = (torch.bfloat16 if kind == "bf16" else torch.float16), (torch.float32 if act == "q8_1" else torch.bfloat16)
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    out, v = mmq.lora(torch.from_numpy(buf).cuda(), torch.from_numpy(A).to(dt).cuda(), torch.from_numpy(B).to(dt).cuda(),
                      torch.from_numpy(scale.astype(np.float32)).cuda(), plan, M, atype=act,
                      base=torch.from_numpy(base).to(io).cuda())
    assert np.array_equal(host(v), wv)
    want = want if act == "q8_1" else rowmodel.bf16(want).astype(np.float64)
    assert np.array_equal(host(out), want)


def test_beside_the_projection(env):
    """The run that it is made for: quantise, plan, the shared projection, the adapters on its
    output in place; against the oracle's projection plus the 64-bit adapters."""
    torch, mmq = env
    import oracle
    M, N, K, R, E = 150, 384, 512, 16, 5
    raw = gen.weights("q4_0", N, K, seed=3, cfg=141)
    xh = gen.act_f32(M, K, seed=4, cfg=141)
    ids = row_ids(M, E, "runs", 6)
    A, B, scale = adapters(torch, "bf16", E, R, K, N, 7)
    packed = mmq.repack_weights("q4_0", torch.from_numpy(raw).cuda(), N, K)
    act = mmq.quantize_act(torch.from_numpy(xh).cuda())
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    out = mmq.gemm("q4_0", packed, act, M, N, K)
    mmq.lora(act, A.cuda(), B.cuda(), scale.cuda(), plan, M, base=out, out=out)
    oracle.build()
    rq, rs, _ = oracle.quantize_q8_1(xh)
    ref = oracle.gemm_f64("q4_0", raw, N, K, rq, rs)
    want = rowmodel.lora(rowmodel.act_values("q8_1", rq, rs), host(A), host(B), host(scale), ids, ref)[0]
    assert np.max(np.abs(host(out) - want)) <= 1e-3 * np.max(np.abs(want))


def test_graph_and_streams(env):
    """Captured once, replayed with other activations, adapters' rows and bases; every replay equals
    the eager call on another stream, and two plans' calls interleaved on two streams do too."""
    torch, mmq = env
    M, N, K, R, E = 77, 300, 256, 32, 6
    A, B, scale = (t.cuda() for t in adapters(torch, "f16", E, R, K, N, 8))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    base = torch.zeros((M, N), device="cuda")
    act = torch.zeros(mmq.act_bytes("q8_1", M, K), dtype=torch.uint8, device="cuda")
    got = {}

    def path(stream=None):
        return mmq.lora(act, A, B, scale, mmq.group_rows(ids, E, stream=stream), M, base=base, stream=stream)
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
        act.copy_(torch.from_numpy(activations(mmq, "q8_1", M, K, 30 + rep)[0]))
        ids.copy_(torch.from_numpy(row_ids(M, E, ["mixed", "runs", "one", "none"][rep], rep)))
        base.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        pairs = [path(s) for s in (s1, s2, s1, s2)]
        torch.cuda.synchronize()
        for out, v in pairs:
            assert torch.equal(out, got["out"][0]) and torch.equal(v, got["out"][1]), rep


def test_binding_refusals(env):
    torch, mmq = env
    M, N, K, R, E = 4, 64, 64, 8, 2
    A, B, scale = (t.cuda() for t in adapters(torch, "bf16", E, R, K, N, 1))
    act = torch.zeros(mmq.act_bytes("q8_1", M, K), dtype=torch.uint8, device="cuda")
    plan = mmq.group_rows(torch.zeros(M, dtype=torch.int32, device="cuda"), E)
    for bad, match in (((act[:-256], A, B, scale, plan, M), "act"), ((act, A.float(), B, scale, plan, M), "adapters"),
                       ((act, A, B.half(), scale, plan, M), "B must"), ((act, A, B[:1], scale, plan, M), "B must"),
                       ((act, A, B, scale[:1], plan, M), "scale"), ((act, A, B, scale.double(), plan, M), "scale"),
                       ((act, A, B, scale, plan, 400), "plan"), ((act.cpu(), A, B, scale, plan, M), "GPU"),
                       ((act, A.transpose(1, 2), B, scale, plan, M), "must")):
        with pytest.raises(ValueError, match=match):
            mmq.lora(*bad)
    with pytest.raises(ValueError, match="base"):
        mmq.lora(act, A, B, scale, plan, M, base=torch.zeros((M, N), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="out"):
        mmq.lora(act, A, B, scale, plan, M, out=torch.zeros((M, N + 1), device="cuda"))
    with pytest.raises(ValueError, match="workspace"):             # one byte, repeated
        mmq.lora(act, A, B, scale, plan, M, workspace=torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20))
    assert mmq.lora_workspace_bytes(E, M, N, K, R) == 0            # few rows: no workspace
    A2, B2, _ = (t.cuda() for t in adapters(torch, "bf16", E, 72, K, N, 1))
    with pytest.raises(mmq.MMQError) as err:
        mmq.lora(act, A2, B2, scale, plan, M, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert err.value.code == mmq.MMQ_EWORKSPACE
    with pytest.raises(mmq.MMQError) as err:                       # a rank that is no multiple of 8
        mmq.lora(act, A[:, :7].contiguous(), B[:, :, :7].contiguous(), scale, plan, M)
    assert err.value.code == mmq.MMQ_EINVAL


def test_a_plan_of_another_batch_stays_inside_the_buffers(env):
    """The entries of a plan made for more rows point past this batch's: the calls hold them inside."""
    torch, mmq = env
    big, N, K, R, E = 3000, 64, 64, 8, 2
    A, B, scale = (t.cuda() for t in adapters(torch, "bf16", E, R, K, N, 1))
    plan = mmq.group_rows(torch.from_numpy(row_ids(big, E, "runs", 1)).cuda(), E)
    for M in (5, 40, 600):
        act = torch.zeros(mmq.act_bytes("q8_1", M, K), dtype=torch.uint8, device="cuda")
        frame = torch.full((M + 64, N), 3.0, device="cuda")
        out, v = mmq.lora(act, A, B, scale, plan, M, base=frame[:M], out=frame[:M])
        dx, dA, dB = mmq.lora_grad(act, A, B, scale, plan, v, out, want_dx=True)
        torch.cuda.synchronize()
        assert bool((frame[M:] == 3.0).all()) and dx.shape == (M, K)


SMALL_SCALED = [(1, 70, 64, 8, 1), (33, 100, 256, 16, 3), (150, 300, 512, 64, 2), (70, 65, 96, 136, 2)]


@pytest.mark.parametrize("act", ["q8_1", "i8_token"])
@pytest.mark.parametrize("kind,ea,eb", [("f16", -24, -24), ("bf16", -60, -50), ("bf16", 40, 50)])
@pytest.mark.parametrize("M,N,K,R,E", SMALL_SCALED)
def test_forward_exact_far_from_one(env, act, kind, ea, eb, M, N, K, R, E):
    """The integers times powers of two: f16 adapters below the smallest normal value (2^-14), bf16
    adapters whose products come near the ends of f32. Nothing rounds but a bf16 output."""
    torch, mmq = env
    print(f"[case] lora scaled {act} {kind} 2^{ea} 2^{eb} M={M} N={N} K={K} R={R} E={E}", flush=True)
    buf, x, A, B = integer_case(mmq, act, kind, M, N, K, R, E, [M, N, K])
    if kind == "f16":
        assert np.abs(A).max() < 2 ** 11 and np.abs(B).max() < 2 ** 10
        A = np.where(np.abs(A) < 1024, A, np.sign(A) * 1023)            # subnormal: below 2^10 units of 2^-24
    A, B = A * np.float32(2.0 ** ea), B * np.float32(2.0 ** eb)
    ids = row_ids(M, E, "mixed", 5)
    scale = 2.0 ** (np.arange(E) % 2) / 2
    want, wv, mag, mag_v = rowmodel.lora(x, A, B, scale, ids, np.zeros((M, N)))
    assert mag_v.max() < 2.0 ** (24 + ea) and (2 * mag).max() < 2.0 ** (25 + ea + eb)
    dt = torch.bfloat16 if kind == "bf16" else torch.float16
    dA, dB = torch.from_numpy(A).to(dt), torch.from_numpy(B).to(dt)
    assert np.array_equal(host(dA), A) and np.array_equal(host(dB), B)
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    out, v = mmq.lora(torch.from_numpy(buf).cuda(), dA.cuda(), dB.cuda(),
                      torch.from_numpy(scale.astype(np.float32)).cuda(), plan, M, atype=act)
    assert np.array_equal(host(v), wv)
    want = want if act == "q8_1" else rowmodel.bf16(want).astype(np.float64)
    assert np.array_equal(host(out), want)


CONTAINED = [("q8_1", "f16", 5, 70, 64, 16, 2), ("q8_1", "bf16", 130, 1100, 128, 72, 3), ("i8_token", "bf16", 150, 301, 512, 64, 2),
             ("i8_token", "f16", 700, 260, 4096, 64, 4), ("q8_1", "bf16", 2300, 130, 64, 72, 3)]


@pytest.mark.parametrize("act,kind,M,N,K,R,E", CONTAINED)
def test_what_is_not_finite_stays_in_its_row(env, act, kind, M, N, K, R, E):
    """A row whose activations' scale or base is not finite changes no other row, nor does what the
    workspace held before."""
    torch, mmq = env
    print(f"[case] lora not finite {act} {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    ids = row_ids(M, E, "runs", 3)
    ids[M // 2] = E - 1
    r = np.random.default_rng([M, N])
    q = r.integers(-127, 128, (M, K)).astype(np.int8)
    q[q == 0] = 1                                                # so that the row's every product is NaN
    s = r.random((M, K // 32) if act == "q8_1" else M).astype(np.float32)
    A, B, scale = (t.cuda() for t in adapters(torch, kind, E, R, K, N, 8))
    io = torch.float32 if act == "q8_1" else torch.bfloat16
    base = torch.randn((M, N), generator=torch.Generator().manual_seed(4)).to(io).cuda()
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    need = mmq.lora_workspace_bytes(E, M, N, K, R)

    def run(scales, b, fill):
        buf = mmq.act_q8_1_pack_host(q, scales) if act == "q8_1" else mmq.act_i8_pack_host(q, scales)
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda") if need else None
        return mmq.lora(torch.from_numpy(buf).cuda(), A, B, scale, plan, M, atype=act, base=b, workspace=ws)
    out, v = run(s, base, 0)
    assert bool(out.isfinite().all()) and bool(v.isfinite().all())
    bad = s.copy()
    bad[M // 2] = np.nan
    badb = base.clone()
    badb[0, N - 1] = float("inf")
    out2, v2 = run(bad, badb, 255)
    keep = torch.ones(M, dtype=torch.bool, device="cuda")
    keep[M // 2] = False
    assert torch.equal(v2[keep], v[keep]) and bool(v2[M // 2].isnan().all())
    assert bool(out2[M // 2].isnan().all())
    out[0, N - 1] = float("inf")                                 # a value added to the base alone
    assert torch.equal(out2[keep], out[keep])


@pytest.mark.parametrize("act,kind,M,N,K,R,E", [
    ("i8_token", "f16", 5, 70, 64, 16, 2), ("q8_1", "bf16", 40, 70, 64, 16, 2), ("i8_token", "bf16", 40, 1030, 96, 64, 3),
    ("i8_token", "bf16", 150, 301, 512, 72, 3), ("q8_1", "f16", 150, 300, 512, 72, 3),
    ("i8_token", "f16", 1100, 130, 64, 72, 3), ("q8_1", "bf16", 1100, 132, 64, 72, 3)])
def test_rows_without_an_adapter_do_not_see_their_activations(env, act, kind, M, N, K, R, E):
    """v = 0 and out = base, whatever such a row's activations hold, in one launch and in two."""
    torch, mmq = env
    print(f"[case] lora away {act} {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    ids = row_ids(M, E, "runs", 3)
    away = [0, M // 2, M - 1]
    ids[away] = [-1, E, -1]
    r = np.random.default_rng([M, N])
    q = r.integers(-127, 128, (M, K)).astype(np.int8)
    s = r.random((M, K // 32) if act == "q8_1" else M).astype(np.float32)
    A, B, scale = (t.cuda() for t in adapters(torch, kind, E, R, K, N, 8))
    io = torch.float32 if act == "q8_1" else torch.bfloat16
    base = torch.randn((M, N), generator=torch.Generator().manual_seed(4)).to(io).cuda()
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)

    def run(scales):
        buf = mmq.act_q8_1_pack_host(q, scales) if act == "q8_1" else mmq.act_i8_pack_host(q, scales)
        return mmq.lora(torch.from_numpy(buf).cuda(), A, B, scale, plan, M, atype=act, base=base)
    out, v = run(s)
    for value in (np.nan, np.inf):
        bad = s.copy()
        bad[away] = value
        out2, v2 = run(bad)
        assert not bool(v2[away].any()) and torch.equal(out2[away], base[away]), value
        assert torch.equal(out2, out) and torch.equal(v2, v), value


def summands(total):
    """(q, a): int8 and f16 values with sum q a = total (below 2^24)."""
    q, a = [], []
    while total >= 127:
        h = np.float16(min(total // 127, 65504))
        if int(h) > total // 127:
            h = np.nextafter(h, np.float16(0))
        q.append(127)
        a.append(h)
        total -= 127 * int(h)
    return q + [1], a + [np.float16(total)]


@pytest.mark.parametrize("M,N,K,R,launches", [(6, 70, 64, 8, 1), (6, 70, 512, 72, 2), (6, 68, 64, 72, 2)])
def test_a_single_product_keeps_f32(env, M, N, K, R, launches):
    """One f16 weight times one v of 24 bits a column, the scale a power of two. Both are exactly the
    sums of their terms and all products of terms are added, the small ones first: only additions
    round. The last is off by at most 2^-23 of the result, those before it by 2^-23 of partial sums
    that are below 2^-6, 2^-7 and far less of it; together below (1 + 2^-4) 2^-23."""
    torch, mmq = env
    print(f"[case] lora one product M={M} N={N} K={K} R={R}", flush=True)
    E, r = M, np.random.default_rng([M, N, K, R])
    assert (mmq.lora_workspace_bytes(E, M, N, K, R) == 0) == (launches == 1)
    V = rowmodel.full_significands(r, M, 24)                       # an adapter a row, of one rank that is not 0
    q, A, at = np.zeros((M, K), np.int8), np.zeros((E, R, K), np.float16), r.integers(0, R, M)
    for m in range(M):
        qm, am = summands(int(V[m]))
        where = r.permutation(K)[:len(qm)]
        q[m, where], A[m, at[m], where] = qm, am
    buf = mmq.act_q8_1_pack_host(q, np.full((M, K // 32), 2.0 ** -23, np.float32))
    B = np.zeros((E, N, R), np.float16)
    b = rowmodel.full_significands(r, (E, N), 11) * 2.0 ** -10
    for m in range(M):
        B[m, :, at[m]] = b[m]
    scale = (2.0 ** (np.arange(E) % 3 - 1)).astype(np.float32)
    plan = mmq.group_rows(torch.arange(M, dtype=torch.int32, device="cuda"), E)
    out, v = mmq.lora(torch.from_numpy(buf).cuda(), torch.from_numpy(A).cuda(), torch.from_numpy(B).cuda(),
                      torch.from_numpy(scale).cuda(), plan, M)
    v64 = V * 2.0 ** -23
    assert np.array_equal(host(v)[np.arange(M), at], v64)
    want = scale[:, None].astype(np.float64) * v64[:, None] * b
    assert np.all(np.abs(host(out) - want) <= (1 + 2.0 ** -4) * U23 * want)


# sizes past the one-launch form, with the parts of K that the first of two launches has
TWO = [
    ("q8_1", "bf16", 10, 128, 16416, 16, 8, "mixed", 8),       # few rows an adapter
    ("i8_token", "f16", 100, 130, 16416, 16, 8, "one", 8),     # all rows with one of several adapters
    ("q8_1", "f16", 100, 260, 8224, 32, 2, "runs", 8), ("i8_token", "bf16", 37, 301, 8224, 40, 3, "mixed", 8),
    ("q8_1", "bf16", 90, 303, 11040, 24, 2, "mixed", 8), ("q8_1", "bf16", 150, 516, 4128, 64, 9, "mixed", 4),
    ("i8_token", "f16", 33, 132, 4128, 64, 3, "one", 8),
    ("q8_1", "f16", 64, 6148, 4096, 32, 32, "mixed", 2), ("i8_token", "bf16", 40, 6150, 4096, 24, 30, "mixed", 2),
    ("q8_1", "bf16", 1100, 4100, 2048, 32, 3, "runs", 1), ("i8_token", "f16", 1030, 4099, 2048, 32, 2, "runs", 1),
    ("q8_1", "f16", 1100, 132, 8224, 64, 3, "mixed", 1), ("i8_token", "bf16", 1040, 260, 16416, 16, 2, "runs", 1)]


def parts_workspace(M, R, S):
    return -(-M * R * (4 * S if S > 1 else 6) // 256) * 256


@pytest.mark.parametrize("act,kind,M,N,K,R,E,how,S", TWO)
def test_forward_in_two_launches(env, act, kind, M, N, K, R, E, how, S):
    assert env[1].lora_workspace_bytes(E, M, N, K, R) == parts_workspace(M, R, S)
    test_forward(env, act, kind, M, N, K, R, E, how)


@pytest.mark.parametrize("case", [TWO[1], TWO[3], TWO[7], TWO[10]])
def test_two_launches_do_not_read_what_the_workspace_held(env, case):
    torch, mmq = env
    act, kind, M, N, K, R, E, how, S = case
    print(f"[case] lora workspace {case}", flush=True)
    ids = row_ids(M, E, how, 1)
    dev = [t.cuda() for t in (torch.from_numpy(activations(mmq, act, M, K, 2)[0]), *adapters(torch, kind, E, R, K, N, 3))]
    plan = mmq.group_rows(torch.from_numpy(ids).cuda(), E)
    need = mmq.lora_workspace_bytes(E, M, N, K, R)
    assert need == parts_workspace(M, R, S)
    want = None
    for fill in (0, 255):                                  # bytes of 255: NaN in f32 and in bf16
        ws = torch.full((need + 64,), fill, dtype=torch.uint8, device="cuda")
        out, v = mmq.lora(*dev, plan, M, atype=act, workspace=ws[:need])
        assert bool((ws[need:] == fill).all())
        if want is not None:
            assert torch.equal(out, want[0]) and torch.equal(v, want[1])
        want = out, v
    assert bool(out.isfinite().all())


def test_two_launches_in_a_graph_and_on_streams(env):
    """As test_graph_and_streams, at sizes that need a workspace: each call's is its own."""
    torch, mmq = env
    M, N, K, R, E = 77, 300, 8224, 32, 6
    assert mmq.lora_workspace_bytes(E, M, N, K, R) == parts_workspace(M, R, 8)
    A, B, scale = (t.cuda() for t in adapters(torch, "f16", E, R, K, N, 8))
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    base = torch.zeros((M, N), device="cuda")
    acts = [torch.zeros(mmq.act_bytes("q8_1", M, K), dtype=torch.uint8, device="cuda") for _ in range(2)]
    got = {}

    def path(act, stream=None):
        return mmq.lora(act, A, B, scale, mmq.group_rows(ids, E, stream=stream), M, base=base, stream=stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        path(acts[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got["out"] = [path(a) for a in acts]
    for rep in range(4):
        for i, a in enumerate(acts):
            a.copy_(torch.from_numpy(activations(mmq, "q8_1", M, K, 30 + 2 * rep + i)[0]))
        ids.copy_(torch.from_numpy(row_ids(M, E, ["mixed", "runs", "one", "none"][rep], rep)))
        base.normal_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        every = [(i, path(acts[i], s)) for i, s in ((0, s1), (1, s2), (1, s1), (0, s2))]
        torch.cuda.synchronize()
        for i, (out, v) in every:
            assert torch.equal(out, got["out"][i][0]) and torch.equal(v, got["out"][i][1]), rep


@pytest.mark.parametrize("act,kind,M,N,K,R,E", [
    ("q8_1", "bf16", 40, 70, 64, 16, 2), ("i8_token", "f16", 40, 68, 64, 16, 2), ("q8_1", "f16", 150, 301, 512, 72, 3),
    ("i8_token", "bf16", 150, 300, 512, 72, 3), ("q8_1", "bf16", 1100, 132, 64, 72, 3), ("i8_token", "f16", 1100, 130, 64, 72, 3)])
def test_rows_without_an_adapter_are_the_base_bit_for_bit(env, act, kind, M, N, K, R, E):
    """In one launch and in two: zeros keep their sign, denormal values and infinities stay."""
    torch, mmq = env
    print(f"[case] lora base bits {act} {kind} M={M} N={N} K={K} R={R} E={E}", flush=True)
    ids = row_ids(M, E, "runs", 3)
    ids[::3] = -1
    away = torch.from_numpy((ids < 0) | (ids >= E)).cuda()
    io, bits = (torch.float32, torch.int32) if act == "q8_1" else (torch.bfloat16, torch.int16)
    A, B, scale = (t.cuda() for t in adapters(torch, kind, E, R, K, N, 8))
    buf = torch.from_numpy(activations(mmq, act, M, K, 2)[0]).cuda()
    base = torch.randn((M, N), generator=torch.Generator().manual_seed(4)).to(io).cuda()
    for i, value in enumerate((-0.0, 0.0, 1e-40, float("inf"), -float("inf"))):
        base[:, i::11] = value
    out, _ = mmq.lora(buf, A, B, scale, mmq.group_rows(torch.from_numpy(ids).cuda(), E), M, atype=act, base=base)
    assert torch.equal(out[away].view(bits), base[away].view(bits))
