"""Host-side tests of the row-group calls (no GPU needed): sizes of the plan and the refusals,
each of which returns before any HIP call, and the binding's own checks."""
import ctypes

import pytest


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


def _up(a, b=256):
    return (a + b - 1) // b * b


@pytest.mark.parametrize("E,T,top_k", [(1, 1, 1), (8, 70, 1), (64, 512, 8), (4096, 3, 2), (4096, 4096, 8), (3, 40000, 3)])
def test_plan_regions(mmq, E, T, top_k):
    P = T * top_k
    U = P // 64 + min(E + 1, P)
    o = mmq.group_region_offsets(E, T, top_k)
    assert o[0] == 0
    assert o[1] == _up(4 * (E + 1))
    assert o[2] == o[1] + _up(4 * P)
    assert o[3] == o[2] + _up(4 * P)
    assert mmq.group_bytes(E, T, top_k) >= o[3] + _up(16 * U)


@pytest.mark.parametrize("E,T,top_k", [(0, 1, 1), (4097, 1, 1), (8, 0, 1), (8, 4, 0), (8, 4, 9), (8, -1, 1),
                                       (8, (1 << 24) + 1, 1), (8, 1 << 22, 5), (8, 1 << 62, 8)])
def test_plan_sizes_refused(mmq, E, T, top_k):
    assert mmq.group_bytes(E, T, top_k) == 0
    with pytest.raises(mmq.MMQError):
        mmq.group_region_offsets(E, T, top_k)
    assert mmq.lib().mmq_group_rows(GOOD, E, T, top_k, GOOD, None) == mmq.MMQ_EINVAL
    assert mmq.lib().mmq_moe_gather(0, GOOD, 64, GOOD, E, T, top_k, 64, GOOD, 64, None) == mmq.MMQ_EINVAL


def test_group_rows_refusals(mmq):
    f = mmq.lib().mmq_group_rows
    assert f(None, 8, 4, 2, GOOD, None) == mmq.MMQ_EINVAL
    assert f(GOOD, 8, 4, 2, None, None) == mmq.MMQ_EINVAL
    assert f(BAD, 8, 4, 2, GOOD, None) == mmq.MMQ_EALIGN
    assert f(GOOD, 8, 4, 2, BAD, None) == mmq.MMQ_EALIGN


def _calls(mmq):
    L = mmq.lib()

    def gather(o=0, x=GOOD, ldx=64, plan=GOOD, N=64, rows=GOOD, ldr=64):
        return L.mmq_moe_gather(o, x, ldx, plan, 8, 4, 2, N, rows, ldr, None)

    def combine(o=0, z=GOOD, ldz=64, r=0, w=GOOD, plan=GOOD, N=64, y=GOOD, ldy=64):
        return L.mmq_moe_combine(o, z, ldz, r, w, plan, 8, 4, 2, N, y, ldy, None)

    def grad(o=0, dy=GOOD, lddy=64, z=GOOD, ldz=64, r=0, w=GOOD, plan=GOOD, N=64, dz=GOOD, lddz=64, dw=GOOD):
        return L.mmq_moe_combine_grad(o, dy, lddy, z, ldz, r, w, plan, 8, 4, 2, N, dz, lddz, dw, None)
    return gather, combine, grad


def test_row_call_refusals(mmq):
    gather, combine, grad = _calls(mmq)
    for f, pointers in ((gather, "x plan rows"), (combine, "z plan y"), (grad, "dy z w plan dz dw")):
        for p in pointers.split():
            assert f(**{p: None}) == mmq.MMQ_EINVAL, p
            assert f(**{p: BAD}) == mmq.MMQ_EALIGN, p
        assert f(N=0) == mmq.MMQ_EINVAL
        assert f(N=(1 << 24) + 1) == mmq.MMQ_EINVAL
        assert f(o=3) == mmq.MMQ_EINVAL
        assert f(o=2) == mmq.MMQ_EUNSUPPORTED
    for f, lds in ((gather, "ldx ldr"), (combine, "ldz ldy"), (grad, "lddy ldz lddz")):
        for ld in lds.split():
            assert f(**{ld: 63}) == mmq.MMQ_EINVAL, ld
    assert combine(w=BAD) == mmq.MMQ_EALIGN
    assert combine(r=2) == mmq.MMQ_EINVAL
    assert grad(r=-1) == mmq.MMQ_EINVAL


def test_binding_refuses_host_tensors(mmq):
    import torch
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        mmq.group_rows(ids, 8)
    plan = torch.zeros(mmq.group_bytes(8, 4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        mmq.moe_gather(torch.zeros(4, 64), plan, 8, 2)
    with pytest.raises(ValueError, match="GPU"):
        mmq.moe_combine(torch.zeros(8, 64), plan, 8, 4, 2)
    with pytest.raises(ValueError, match="GPU"):
        mmq.moe_combine_grad(torch.zeros(4, 64), torch.zeros(8, 64), plan, 8, 2, torch.zeros(4, 2))


def test_binding_refuses_another_gpus_stream(mmq):
    class Stream:
        cuda_stream = 0
        device_index = 1
    with pytest.raises(ValueError, match="stream"):
        mmq._raw_stream(Stream, 0)
    assert mmq._raw_stream(Stream, 1) == 0


def test_binding_refuses_rows_and_orders_it_does_not_know(mmq):
    import torch
    assert mmq._pair_rows("f", torch.zeros(4, 2, 64), 8).shape == (8, 64)
    assert mmq._pair_rows("f", torch.zeros(4, 2, 70)[:, :, :64], 8).stride() == (70, 1)
    for z in (torch.zeros(2, 4, 64).transpose(0, 1), torch.zeros(4, 3, 64)[:, :2], torch.zeros(64), torch.zeros(9, 64)):
        with pytest.raises(ValueError, match="pairs' rows"):
            mmq._pair_rows("f", z, 8)
    assert [mmq._row_order("f", r) for r in ("pair", "sorted")] == [0, 1]
    for r in ("expert", "", None, 2):
        with pytest.raises(ValueError, match="order"):
            mmq._row_order("f", r)
