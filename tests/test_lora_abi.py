"""Host-side tests of the adapters' calls (no GPU needed): workspace sizes and refusals, each of
which returns before any HIP call."""
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

SIZES_REFUSED = [dict(E=0), dict(E=4097), dict(M=0), dict(M=(1 << 24) + 1), dict(K=0), dict(K=48), dict(K=1 << 24),
                 dict(R=0), dict(R=4), dict(R=12), dict(R=264), dict(M=1 << 24, K=1 << 23)]


@pytest.mark.parametrize("bad", SIZES_REFUSED)
def test_workspace_sizes_refused(mmq, bad):
    k = dict(E=4, M=4000, N=4096, K=4096, R=64)
    assert mmq.lora_workspace_bytes(**k) >= 4000 * 64 * 4
    k.update(bad)
    assert mmq.lora_workspace_bytes(**k) == 0


def _lora(mmq, a=0, act=GOOD, d=0, A=GOOD, B=GOOD, scale=GOOD, E=4, R=64, plan=GOOD, M=4000, N=4096, K=4096, base=GOOD,
          ldb=4096, out=GOOD, ldo=4096, v=GOOD, ws=GOOD, nbytes=None):
    if nbytes is None:
        nbytes = mmq.lora_workspace_bytes(E, M, N, K, R) - 1      # one short: nothing is ever enqueued
    return mmq.lib().mmq_lora(a, act, d, A, B, scale, E, R, plan, M, N, K, base, ldb, out, ldo, v, ws, max(nbytes, 0), None)


def test_lora_refusals(mmq):
    assert _lora(mmq) == mmq.MMQ_EWORKSPACE
    assert _lora(mmq, ws=None, nbytes=1 << 30) == mmq.MMQ_EWORKSPACE
    assert _lora(mmq, ws=BAD, nbytes=1 << 30) == mmq.MMQ_EALIGN
    for p in "act A B scale plan out v".split():
        assert _lora(mmq, **{p: None}) == mmq.MMQ_EINVAL, p
        assert _lora(mmq, **{p: BAD}) == mmq.MMQ_EALIGN, p
    assert _lora(mmq, base=BAD) == mmq.MMQ_EALIGN
    for bad in SIZES_REFUSED + [dict(a=2), dict(a=-1), dict(d=2), dict(N=0), dict(N=4097), dict(ldb=4095),
                                dict(ldo=4095), dict(ldb=4097), dict(N=1 << 24, M=1 << 24, ldb=1 << 24, ldo=1 << 24)]:
        assert _lora(mmq, **bad) == mmq.MMQ_EINVAL, bad
    # a base of another stride is fine unless it is the output itself; no base needs no stride
    assert _lora(mmq, base=ctypes.c_void_p(0x20000), ldb=4097) == mmq.MMQ_EWORKSPACE
    assert _lora(mmq, base=None, ldb=0) == mmq.MMQ_EWORKSPACE


GRAD_REFUSED = [dict(E=0), dict(M=0), dict(K=48), dict(R=12), dict(R=264), dict(N=0), dict(E=4096, N=1 << 18),
                dict(E=4096, K=1 << 18)]


@pytest.mark.parametrize("bad", GRAD_REFUSED)
def test_grad_workspace_sizes_refused(mmq, bad):
    k = dict(E=4, M=100, N=64, K=512, R=16)
    assert mmq.lora_grad_workspace_bytes(**k) >= 2 * 100 * 16 * 4
    k.update(bad)
    assert mmq.lora_grad_workspace_bytes(**k) == 0


def _grad(mmq, a=0, act=GOOD, d=0, A=GOOD, B=GOOD, scale=GOOD, E=4, R=16, plan=GOOD, M=100, N=64, K=512, v=GOOD,
          dy=GOOD, lddy=None, dx_base=GOOD, ldxb=512, dx=GOOD, lddx=512, dA=GOOD, dB=GOOD, ws=GOOD, nbytes=None):
    if nbytes is None:
        nbytes = mmq.lora_grad_workspace_bytes(E, M, N, K, R) - 1
    return mmq.lib().mmq_lora_grad(a, act, d, A, B, scale, E, R, plan, M, N, K, v, dy, N if lddy is None else lddy,
                                   dx_base, ldxb, dx, lddx, dA, dB, ws, max(nbytes, 0), None)


def test_lora_grad_refusals(mmq):
    assert _grad(mmq) == mmq.MMQ_EWORKSPACE
    assert _grad(mmq, ws=None, nbytes=1 << 30) == mmq.MMQ_EWORKSPACE
    assert _grad(mmq, ws=BAD, nbytes=1 << 30) == mmq.MMQ_EALIGN
    for p in "act A B scale plan v dy dA dB".split():
        assert _grad(mmq, **{p: None}) == mmq.MMQ_EINVAL, p
        assert _grad(mmq, **{p: BAD}) == mmq.MMQ_EALIGN, p
    assert _grad(mmq, dx=BAD) == mmq.MMQ_EALIGN
    assert _grad(mmq, dx_base=BAD) == mmq.MMQ_EALIGN
    for bad in GRAD_REFUSED + [dict(a=2), dict(d=-1), dict(lddy=63), dict(ldxb=511), dict(lddx=511), dict(lddx=513)]:
        assert _grad(mmq, **bad) == mmq.MMQ_EINVAL, bad
    # without dx its strides do not matter; without a base its stride does not
    assert _grad(mmq, dx=None, lddx=0, ldxb=0) == mmq.MMQ_EWORKSPACE
    assert _grad(mmq, dx_base=None, ldxb=0) == mmq.MMQ_EWORKSPACE
