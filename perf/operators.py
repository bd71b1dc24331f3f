"""Cases and plain forms of the operators around the shared projection and the expert products.

Three operators, each on the buffers that the quantised products read and write:

* lora, lora_grad - low-rank adapters of many requests beside a shared projection, and their
  gradients taken from the 8-bit activations (the act buffer kept as the checkpoint):
      v = x^ A_e^T;  out = base + s_e v B_e^T          (e: the row's adapter, or none)
      u = s_e dy B_e;  dB_e = s_e dy^T v;  dA_e = u^T x^;  dx = dx_base + u A_e
* dispatch - (token, slot) pairs sorted by expert: the plan, and the tokens' rows in its order
* combine, combine_grad - the experts' rows weighted and summed back into tokens, and the
  gradients for the rows and the weights

The state holds what a program has before the call: the act buffer in its documented layout, the
adapters, the plan of the batch (kept for all projections of a step), outputs of earlier calls.
"""
import math

import torch

own = False

UNIT = 64           # rows of a plan's unit at most
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------------- the cases

def listed():
    lora = lambda name, **k: dict(name=name, op="lora", **k)          # noqa: E731
    grad = lambda name, **k: dict(name=name, op="lora_grad", **k)     # noqa: E731
    return [
        # one token of one request at a 7B attention projection: latency
        lora("lora_decode_1", act="q8_1", adapter="bf16", M=1, N=4096, K=4096, R=16, E=8, rows="mixed"),
        # a decode batch: 64 requests, 32 adapters, the up projection
        lora("lora_decode_64", act="q8_1", adapter="f16", M=64, N=14336, K=4096, R=32, E=32, rows="mixed"),
        # a prefill batch of several requests, each with its adapter
        lora("lora_prefill_2048", act="q8_1", adapter="bf16", M=2048, N=4096, K=4096, R=64, E=8, rows="runs"),
        # the per-channel W8A8 projection's share of a tensor-parallel group, ragged
        lora("lora_w8a8_517", act="i8_token", adapter="f16", M=517, N=1536, K=4096, R=24, E=6, rows="runs"),
        # a training step of adapters on a frozen quantised projection
        grad("grad_2048", act="q8_1", adapter="bf16", M=2048, N=4096, K=4096, R=16, E=4, rows="runs"),
        # the same beside the W8A8 down projection, odd sizes, bf16 gradients
        grad("grad_w8a8_331", act="i8_token", adapter="f16", M=331, N=1003, K=11008, R=40, E=3, rows="runs"),
        # a decode step of a 64-expert layer, 8 experts a token
        dict(name="dispatch_10", op="dispatch", dtype="f32", T=10, top_k=8, E=64, N=4096, away=0.0),
        # a long prompt; a quarter of the pairs goes to experts that another rank holds
        dict(name="dispatch_2048", op="dispatch", dtype="bf16", T=2048, top_k=8, E=64, N=4096, away=0.25),
        # the expert products' own output (pair order), back into tokens
        dict(name="combine_512", op="combine", dtype="f32", T=512, top_k=8, E=64, N=2048, order="pair", away=0.0),
        # rows in expert order, ragged, some tokens without an expert here
        dict(name="combine_1999", op="combine", dtype="bf16", T=1999, top_k=2, E=8, N=4100, order="sorted", away=0.5),
        dict(name="combine_grad_512", op="combine_grad", dtype="f32", T=512, top_k=8, E=64, N=2048, order="pair", away=0.0),
        dict(name="combine_grad_77", op="combine_grad", dtype="bf16", T=77, top_k=4, E=16, N=1001, order="sorted", away=0.25),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_grad", "dispatch", "combine", "combine_grad"])
    if op in ("lora", "lora_grad"):
        E = _log(rng, 1, 48)
        R = 8 * rng.randint(1, min(16, max(1, 128 // E)))
        M = _log(rng, 1 if op == "lora" else 16, 2048)
        N, K = _log(rng, 64, 14336), 32 * _log(rng, 2, 448)
        N, K = min(N, 2048 * 4096 // M), min(K, 2048 * 4096 // M // 32 * 32)
        if op == "lora_grad":
            R = min(R, 64)
        return dict(op=op, act=rng.choice(["q8_1", "i8_token"]), adapter=rng.choice(["bf16", "f16"]),
                    M=M, N=N, K=K, R=R, E=E, rows=rng.choice(["mixed", "runs"]))
    T, E = _log(rng, 1, 2048), _log(rng, 1, 128)
    top_k = rng.randint(1, min(8, E))
    N = _log(rng, 32, 8192)
    limit = 2048 * 8 * 4096 // (2 if op == "dispatch" else 8)     # the largest listed case's values
    N = max(1, min(N, limit // (T * top_k)))
    c = dict(op=op, dtype=rng.choice(["f32", "bf16"]), T=T, top_k=top_k, E=E, N=N,
             away=rng.choice([0.0, 0.1, 0.5]))
    if op != "dispatch":
        c["order"] = rng.choice(["pair", "sorted"])
    return c


# ------------------------------------------------------------------------------- the inputs

def _up(a, b):
    return (a + b - 1) // b * b


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda") * std


def _bytes(t, size):
    """t's bytes, padded with zeros to `size`."""
    b = t.contiguous().view(-1).view(torch.uint8)
    return torch.cat([b, b.new_zeros(size - b.numel())])


def _tiled(t, Mp, KBp):
    """[M, KB] per row and block -> tile-major [Mp/32][KBp][32]."""
    full = t.new_zeros(Mp, KBp)
    full[:t.shape[0], :t.shape[1]] = t
    return full.view(Mp // 32, 32, KBp).transpose(1, 2)


def _act(g, kind, M, K):
    """An act buffer of N(0,1) activations with 0.1% outliers x20."""
    x = _normal(g, (M, K))
    x = torch.where(torch.rand((M, K), generator=g, device="cuda") < 1e-3, x * 20, x)
    KB, Mp = K // 32, _up(M, 32)
    KBp = _up(KB, 8)
    amax = x.view(M, KB, 32).abs().amax(2) if kind == "q8_1" else x.abs().amax(1, keepdim=True)
    d = amax / 127
    per = d.repeat_interleave(32, 1) if kind == "q8_1" else d
    q = (x * (1 / per)).round().clamp(-128, 127).to(torch.int8)
    full = q.new_zeros(Mp, KBp * 32)
    full[:M, :K] = q
    parts = [_bytes(full.view(Mp // 32, 32, KBp, 2, 16).permute(0, 2, 3, 1, 4), Mp * KBp * 32)]
    if kind == "i8_token":
        sa = d.new_zeros(Mp)
        sa[:M] = d[:, 0]
        return torch.cat(parts + [_bytes(sa, _up(Mp * 4, 256))])
    xs = d.half()
    grp = q.view(M, KB, 4, 8).sum(3, dtype=torch.int32)
    bits = xs.view(torch.int16).int() & 0xFFFF
    cells = Mp * KBp * 4
    parts.append(_bytes(_tiled(bits | (bits << 16), Mp, KBp), _up(cells, 256)))
    parts.append(_bytes(_tiled(xs.float() * grp.sum(2), Mp, KBp), _up(cells, 256)))
    gh = (grp.float() * 2.0 ** -13).half().view(torch.int16).int() & 0xFFFF
    pair = [_tiled(gh[..., 2 * h] | (gh[..., 2 * h + 1] << 16), Mp, KBp) for h in (0, 1)]
    parts.append(_bytes(torch.stack(pair, 2), _up(2 * cells, 256)))
    return torch.cat(parts)


def _plan(ids, E):
    """The plan of ids [T, top_k] in its documented layout, as int32 words."""
    flat = ids.reshape(-1).long()
    P = flat.numel()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    order = torch.sort(key, stable=True).indices
    count = torch.bincount(key, minlength=E + 1)
    end = count.cumsum(0)
    pos = torch.empty_like(flat)
    pos[order] = torch.arange(P, device=flat.device)
    pos = torch.where(key < E, pos, -1)
    units = P // UNIT + min(E + 1, P)
    last = ((count + UNIT - 1) // UNIT).cumsum(0)
    u = torch.arange(units, device=flat.device)
    grp = torch.searchsorted(last, u, right=True).clamp(max=E)
    nth = u - (last - (count + UNIT - 1) // UNIT)[grp]
    left = (count[grp] - UNIT * nth).clamp(0, UNIT)
    unit = torch.stack([grp, (end - count)[grp] + UNIT * nth, left, torch.zeros_like(u)], 1)
    unit = torch.where((left > 0)[:, None], unit, 0)
    words = [torch.cat([end.new_zeros(1), end[:E]]), order, pos, unit.reshape(-1)]
    return torch.cat([_bytes(w.int(), _up(w.numel() * 4, 256)) for w in words])


def _row_ids(g, case):
    """The rows' adapters: requests mixed row by row (decode), or runs of rows (prefill); every
    ninth row or run has none."""
    M, E = case["M"], case["E"]
    perm = torch.randperm(E, generator=g, device="cuda")
    if case["rows"] == "mixed":
        which = torch.arange(M, device="cuda")
    else:
        cut = torch.rand((M,), generator=g, device="cuda") < min(1.0, (E - 1) / M)
        cut[0] = False
        which = cut.cumsum(0)
    return torch.where(which % 9 == 8, -1, perm[which % E]).int()


def _pair_ids(g, case):
    """Each token's distinct experts; a share of the pairs goes to experts held elsewhere."""
    T, E, k = case["T"], case["E"], case["top_k"]
    ids = torch.rand((T, E), generator=g, device="cuda").argsort(1)[:, :k].int()
    away = torch.rand((T, k), generator=g, device="cuda") < case["away"]
    return torch.where(away, -1, ids)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    s = dict(case=dict(case), op=case["op"])
    if case["op"] in ("lora", "lora_grad"):
        M, N, K, R, E = (case[k] for k in "MNKRE")
        io = DT["f32" if case["act"] == "q8_1" else "bf16"]
        s["act"] = _act(g, case["act"], M, K)
        s["A"] = _normal(g, (E, R, K), K ** -0.5).to(DT[case["adapter"]])
        s["B"] = _normal(g, (E, N, R), 0.3 * R ** -0.5).to(DT[case["adapter"]])
        s["scale"] = 0.5 + 1.5 * torch.rand((E,), generator=g, device="cuda")
        s["ids"] = _row_ids(g, case)
        s["plan"] = _plan(s["ids"], E)
        if case["op"] == "lora":
            s["base"] = _normal(g, (M, N)).to(io)
        else:
            x, e = _values(s["act"], case["act"], M, K), s["ids"].long()
            v = (x.double() @ s["A"].double().reshape(E * R, K).T).view(M, E, R)
            v = v[torch.arange(M, device="cuda"), e.clamp(min=0)].float()
            s["v"] = torch.where(e[:, None] >= 0, v, 0.0)
            s["dy"] = _normal(g, (M, N), 0.05).to(io)
            s["dx_base"] = _normal(g, (M, K), 0.05)
        return s
    T, N, E, k = case["T"], case["N"], case["E"], case["top_k"]
    dt = DT[case["dtype"]]
    s["ids"] = _pair_ids(g, case)
    if case["op"] == "dispatch":
        s["x"] = _normal(g, (T, N)).to(dt)
        s["rows"] = torch.zeros((T * k, N), dtype=dt, device="cuda")
        return s
    s["plan"] = _plan(s["ids"], E)
    s["w"] = _normal(g, (T, k)).softmax(1)
    z = _normal(g, (T * k, N)).to(dt)
    there = s["ids"].view(-1) >= 0
    if case["order"] == "sorted":
        there = there.sort(descending=True, stable=True).values
    s["z"] = torch.where(there[:, None], z, float("nan"))     # the products left these rows unwritten
    if case["op"] == "combine_grad":
        s["dy"] = _normal(g, (T, N), 0.05).to(dt)
        s["dz"] = torch.zeros((T * k, N), dtype=dt, device="cuda")
    return s


# ------------------------------------------------------------------------------- plain forms

def _values(act, kind, M, K):
    """x^ [M, K] in f32 from an act buffer (exact: an 11-bit scale, or one rounding with the f32
    per-token scale, times 8 bits)."""
    Mp, KBp = _up(M, 32), _up(K // 32, 8)
    n = Mp * KBp * 32
    q = act[:n].view(torch.int8).view(Mp // 32, KBp, 2, 32, 16).permute(0, 3, 1, 2, 4)
    at = _up(n, 256)
    if kind == "i8_token":
        return q.reshape(Mp, -1)[:M, :K].float() * act[at:at + 4 * Mp].view(torch.float32)[:M, None]
    xs = act[at:at + 4 * Mp * KBp].view(torch.float16).view(Mp // 32, KBp, 32, 2)[..., 0]
    x = q.reshape(Mp, KBp, 32).float() * xs.transpose(1, 2).reshape(Mp, KBp, 1).float()
    return x.view(Mp, -1)[:M, :K]


def _mask(s):
    """[M, E]: the row's scale at its adapter, 0 elsewhere; and the same with 1."""
    E = s["case"]["E"]
    hit = s["ids"][:, None] == torch.arange(E, device="cuda", dtype=torch.int32)
    return hit.float() * s["scale"], hit


def _plain_lora(s):
    c = s["case"]
    M, N, K, R, E = (c[k] for k in "MNKRE")
    scale, hit = _mask(s)
    x = _values(s["act"], c["act"], M, K)
    every = (x @ s["A"].float().view(E * R, K).T).view(M, E, R) * hit[:, :, None]
    flat = s["B"].float().permute(0, 2, 1).reshape(E * R, N)
    out = s["base"].float() + (every * scale[:, :, None]).view(M, E * R) @ flat
    return {"out": out.to(s["base"].dtype), "v": every.sum(1)}


def _plain_lora_grad(s):
    c = s["case"]
    M, N, K, R, E = (c[k] for k in "MNKRE")
    scale, hit = _mask(s)
    x, dy = _values(s["act"], c["act"], M, K), s["dy"].float()
    flat = s["B"].float().permute(0, 2, 1).reshape(E * R, N)
    u = ((dy @ flat.T).view(M, E, R) * scale[:, :, None]).view(M, E * R)
    dx = s["dx_base"] + u @ s["A"].float().view(E * R, K)
    dA = (u.T @ x).view(E, R, K)
    v = (s["v"][:, None, :] * scale[:, :, None]).view(M, E * R)
    return {"dx": dx, "dA": dA, "dB": (dy.T @ v).view(N, E, R).permute(1, 0, 2).contiguous()}


def _plain_sort(s):
    E, k = s["case"]["E"], s["case"]["top_k"]
    flat = s["ids"].view(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, E)
    sorted_key, order = torch.sort(key, stable=True)
    offs = (key[:, None] < torch.arange(E + 1, device="cuda")).sum(0)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    rows = torch.where((sorted_key < E)[:, None], s["x"][order // k], 0)
    return {"offs": offs.int(), "order": order.int(), "pos": torch.where(key < E, pos, -1).int(), "rows": rows}


def _pair_rows(s):
    """Each pair's row of z and whether it has one."""
    c = s["case"]
    P = c["T"] * c["top_k"]
    words = s["plan"].view(torch.int32)
    at = (_up((c["E"] + 1) * 4, 256) + _up(P * 4, 256)) // 4
    pos = words[at:at + P].long()
    row = pos if c["order"] == "sorted" else torch.arange(P, device="cuda")
    return row.clamp(min=0), pos >= 0


def _plain_combine(s):
    c = s["case"]
    row, has = _pair_rows(s)
    z = torch.where(has[:, None], s["z"][row].float(), 0.0).view(c["T"], c["top_k"], c["N"])
    return {"y": (z * s["w"][:, :, None]).sum(1).to(s["z"].dtype)}


def _plain_combine_grad(s):
    c = s["case"]
    row, has = _pair_rows(s)
    dy = s["dy"].float().repeat_interleave(c["top_k"], 0)
    dw = torch.where(has, (dy * s["z"][row].float()).sum(1), 0.0).view(c["T"], c["top_k"])
    dz = torch.zeros_like(s["z"])
    keep = torch.nonzero(has)[:, 0]
    dz[row[keep]] = (dy * s["w"].view(-1, 1))[keep].to(dz.dtype)
    return {"dz": dz, "dw": dw}


# --------------------------------------------------------------------------- the operators

def _own(s):
    import block_quantized_int8_amd as mmq
    c = s["case"]
    if c["op"] == "lora":
        out, v = mmq.lora(s["act"], s["A"], s["B"], s["scale"], s["plan"], c["M"], atype=c["act"], base=s["base"])
        return {"out": out, "v": v}
    if c["op"] == "lora_grad":
        dx, dA, dB = mmq.lora_grad(s["act"], s["A"], s["B"], s["scale"], s["plan"], s["v"], s["dy"],
                                   atype=c["act"], dx_base=s["dx_base"])
        return {"dx": dx, "dA": dA, "dB": dB}
    E, T, k = c["E"], c["T"], c["top_k"]
    if c["op"] == "dispatch":
        plan = mmq.group_rows(s["ids"], E)
        rows = mmq.moe_gather(s["x"], plan, E, k, out=s["rows"])
        offs, order, pos, _ = mmq.group_views(plan, E, T, k)
        return {"offs": offs, "order": order, "pos": pos, "rows": rows}
    if c["op"] == "combine":
        return {"y": mmq.moe_combine(s["z"], s["plan"], E, T, k, weights=s["w"], order=c["order"])}
    dz, dw = mmq.moe_combine_grad(s["dy"], s["z"], s["plan"], E, k, s["w"], order=c["order"], dz=s["dz"])
    return {"dz": dz, "dw": dw}


_PLAIN = {"lora": _plain_lora, "lora_grad": _plain_lora_grad, "dispatch": _plain_sort,
          "combine": _plain_combine, "combine_grad": _plain_combine_grad}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------ in 64 bits

def _exact_values(act, kind, M, K):
    """x^ from the layout's own formulas: the byte of (m, k) and the scale of (m, k / 32)."""
    KBp, Mp = _up(K // 32, 8), _up(M, 32)
    m = torch.arange(M, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None, :]
    at = ((m // 32) * KBp + k // 32) * 1024 + ((k % 32 // 16) * 32 + m % 32) * 16 + k % 16
    q = act.view(torch.int8)[at].double()
    start = _up(Mp * KBp * 32, 256)
    if kind == "i8_token":
        return q * act[start:].view(torch.float32)[:M].double()[:, None]
    half = act[start:].view(torch.float16)
    b = torch.arange(K // 32, device="cuda")[None, :]
    return q * half[2 * (((m // 32) * KBp + b) * 32 + m % 32)].double().repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("lora", "lora_grad"):
        M, N, K, R, E = (case[k] for k in "MNKRE")
        x = _exact_values(s["act"], case["act"], M, K)
        if case["op"] == "lora":
            out, v = s["base"].double(), x.new_zeros(M, R)
            for e in range(E):
                at = torch.nonzero(s["ids"] == e)[:, 0]
                v[at] = x[at] @ s["A"][e].double().T
                out[at] += s["scale"][e].double() * (v[at] @ s["B"][e].double().T)
            return {"out": out, "v": v}
        dy, dx = s["dy"].double(), s["dx_base"].double()
        dA, dB = x.new_zeros(E, R, K), x.new_zeros(E, N, R)
        for e in range(E):
            at = torch.nonzero(s["ids"] == e)[:, 0]
            u = s["scale"][e].double() * (dy[at] @ s["B"][e].double())
            dx[at] += u @ s["A"][e].double()
            dA[e] = u.T @ x[at]
            dB[e] = s["scale"][e].double() * (dy[at].T @ s["v"][at].double())
        return {"dx": dx, "dA": dA, "dB": dB}
    T, k, N, E = case["T"], case["top_k"], case["N"], case["E"]
    ids = s["ids"].view(-1)
    there = torch.nonzero((ids >= 0) & (ids < E))[:, 0]
    by = there[torch.argsort(ids[there].long() * (T * k) + there)]        # expert order, stable
    if case["op"] == "dispatch":
        rest = torch.nonzero((ids < 0) | (ids >= E))[:, 0]
        pos = torch.full_like(ids, -1)
        pos[by] = torch.arange(by.numel(), device="cuda", dtype=torch.int32)
        rows = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
        rows[:by.numel()] = s["x"].double()[by // k]
        offs = torch.stack([(ids[there] < e).sum() for e in range(E + 1)])
        return {"offs": offs.int(), "order": torch.cat([by, rest]).int(), "pos": pos, "rows": rows}
    z = s["z"].double()
    mine = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")   # the pairs' rows
    mine[by] = z[:by.numel()] if case["order"] == "sorted" else z[by]
    w = s["w"].double().view(-1)
    if case["op"] == "combine":
        y = torch.zeros((T, N), dtype=torch.float64, device="cuda")
        return {"y": y.index_add(0, by // k, mine[by] * w[by, None])}
    dy = s["dy"].double()
    dz = torch.zeros((T * k, N), dtype=torch.float64, device="cuda")
    given = dy[by // k] * w[by, None]
    if case["order"] == "sorted":
        dz[:by.numel()] = given
    else:
        dz[by] = given
    dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
    dw[by] = (mine[by] * dy[by // k]).sum(1)
    return {"dz": dz, "dw": dw.view(T, k)}


# ------------------------------------------------------------------------------------ work

def work(case):
    if case["op"] in ("lora", "lora_grad"):
        M, N, K, R, E = (case[k] for k in "MNKRE")
        used = min(E, M)
        io = 4 if case["act"] == "q8_1" else 2
        act = M * K + (M * (K // 32) * 2 if case["act"] == "q8_1" else 4 * M)
        adapters = used * R * (K + N) * 2 + 4 * E + 4 * M
        if case["op"] == "lora":
            return {"bytes": act + adapters + 2 * M * N * io + 4 * M * R, "flops": 2 * M * R * (K + N)}
        return {"bytes": act + adapters + M * N * io + 4 * M * R + 8 * M * K + 4 * E * R * (K + N),
                "flops": 4 * M * R * (K + N)}
    T, k, N = case["T"], case["top_k"], case["N"]
    size, P = (4 if case["dtype"] == "f32" else 2), T * k
    here = P * (1 - case["away"])
    if case["op"] == "dispatch":
        return {"bytes": 12 * P + 4 * (case["E"] + 1) + (T + here) * N * size, "flops": 0}
    if case["op"] == "combine":
        return {"bytes": (here + T) * N * size + 8 * P, "flops": 2 * here * N}
    return {"bytes": (2 * here + T) * N * size + 12 * P, "flops": 3 * here * N}
