"""Refusals of the 4-bit GEMV, balance and sampling entry points, on the CPU:
bad arguments return the documented status before anything is launched (no
pointer is dereferenced)."""
import ctypes

import pytest

from lfsr_seeded_moe_b200 import nslm

A = 0x10000000  # an aligned address that nothing reads


def _q4(N=64, K=256, group=64, q=A, scales=A + 0x100000, biases=A + 0x200000):
    return nslm.nslm_q4_matrix(q, scales, biases, N, K, group)


@pytest.mark.parametrize("W,kw,want", [
    (_q4(group=16), {}, nslm.NSLM_ERR_SHAPE),
    (_q4(group=0), {}, nslm.NSLM_ERR_SHAPE),
    (_q4(K=96), {}, nslm.NSLM_ERR_SHAPE),            # not a multiple of the group
    (_q4(K=0), {}, nslm.NSLM_ERR_SHAPE),
    (_q4(N=-1), {}, nslm.NSLM_ERR_SHAPE),
    (_q4(q=0), {}, nslm.NSLM_ERR_ARG),
    (_q4(scales=0), {}, nslm.NSLM_ERR_ARG),
    (_q4(q=A + 8), {}, nslm.NSLM_ERR_ALIGN),
    (_q4(scales=A + 2), {}, nslm.NSLM_ERR_ALIGN),
    (_q4(biases=A + 2), {}, nslm.NSLM_ERR_ALIGN),
    (_q4(), dict(M=0), nslm.NSLM_ERR_SHAPE),
    (_q4(), dict(M=9), nslm.NSLM_ERR_SHAPE),
    (_q4(K=16384), dict(M=5), nslm.NSLM_ERR_SHAPE),  # activations exceed shared memory
    (_q4(), dict(x=0), nslm.NSLM_ERR_ARG),
    (_q4(), dict(y=0), nslm.NSLM_ERR_ARG),
    (_q4(), dict(x=A + 2), nslm.NSLM_ERR_ALIGN),
    (_q4(), dict(y=A + 4), nslm.NSLM_ERR_ALIGN),
    (_q4(), dict(flags=2), nslm.NSLM_ERR_ARG),
    (None, {}, nslm.NSLM_ERR_ARG),
])
def test_q4_gemv_refusals(W, kw, want):
    a = dict(x=A + 0x300000, M=1, y=A + 0x400000, flags=0)
    a.update(kw)
    rc = nslm.raw().nslm_q4_gemv(None if W is None else ctypes.byref(W), a["x"], a["M"], a["y"], a["flags"], 0)
    assert rc == want
    assert nslm.nslm_last_launch_count() == 0


def _balance(**kw):
    a = dict(logits=A, ids=A, mask=0, T=4, E=8, k=2, counts=A, offsets=0, mean_p=0, loss=A, ws=0, wsb=0)
    a.update(kw)
    return nslm.raw().nslm_moe_balance(a["logits"], a["ids"], a["mask"], a["T"], a["E"], a["k"], 0.01, a["counts"],
                                       a["offsets"], a["mean_p"], a["loss"], a["ws"], a["wsb"], 0)


def test_balance_refusals():
    for kw in (dict(logits=0), dict(ids=0), dict(counts=0), dict(loss=0)):
        assert _balance(**kw) == nslm.NSLM_ERR_ARG, kw
    for kw in (dict(T=-1), dict(k=0), dict(k=9, E=16), dict(E=1), dict(E=1025),
               dict(T=2**28 + 1), dict(T=2**28, k=8)):
        assert _balance(**kw) == nslm.NSLM_ERR_SHAPE, kw
    for name in ("logits", "ids", "mask", "counts", "offsets", "mean_p", "loss"):
        assert _balance(**{name: A + 4}) == nslm.NSLM_ERR_ALIGN, name
    need = nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, 5000, 8, 0, 0, 2)
    assert need > 0
    assert _balance(T=5000) == nslm.NSLM_ERR_WORKSPACE
    assert _balance(T=5000, ws=A, wsb=need - 1) == nslm.NSLM_ERR_WORKSPACE
    assert _balance(T=5000, ws=A + 8, wsb=need) == nslm.NSLM_ERR_ALIGN
    assert nslm.nslm_workspace_bytes(nslm.NSLM_OP_MOE_BALANCE, 1024, 8, 0, 0, 2) == 0
    assert nslm.nslm_last_launch_count() == 0


def test_balance_grad_refusals():
    def call(**kw):
        a = dict(logits=A, counts=A, mask=0, T=4, E=8, k=2, dloss=0, dlogits=A)
        a.update(kw)
        return nslm.raw().nslm_moe_balance_grad(a["logits"], a["counts"], a["mask"], a["T"], a["E"], a["k"], 0.01,
                                                a["dloss"], a["dlogits"], 0)

    for kw in (dict(logits=0), dict(counts=0), dict(dlogits=0)):
        assert call(**kw) == nslm.NSLM_ERR_ARG, kw
    for kw in (dict(T=-1), dict(k=0), dict(k=9, E=16), dict(E=1), dict(E=1025),
               dict(T=2**28 + 1), dict(T=2**28, k=8)):
        assert call(**kw) == nslm.NSLM_ERR_SHAPE, kw
    for name in ("logits", "counts", "mask", "dloss", "dlogits"):
        assert call(**{name: A + 4}) == nslm.NSLM_ERR_ALIGN, name
    assert nslm.nslm_last_launch_count() == 0


def test_sample_refusals():
    def call(params=None, **kw):
        a = dict(logits=A, type=0, B=2, V=100, ld=100, u=A, token=A, prob=0)
        a.update(kw)
        return nslm.raw().nslm_sample(a["logits"], a["type"], a["B"], a["V"], a["ld"],
                                      None if params is None else ctypes.byref(params), a["u"], a["token"], a["prob"], 0)

    for kw in (dict(logits=0), dict(u=0), dict(token=0), dict(type=2), dict(type=-1)):
        assert call(**kw) == nslm.NSLM_ERR_ARG, kw
    for kw in (dict(B=-1), dict(V=0), dict(V=262145, ld=262145), dict(ld=99), dict(B=2**24 + 1)):
        assert call(**kw) == nslm.NSLM_ERR_SHAPE, kw
    for name in ("logits", "u", "token", "prob"):
        assert call(**{name: A + 4}) == nslm.NSLM_ERR_ALIGN, name
    for name in ("temperature", "top_k", "top_p", "min_p"):
        assert call(params=nslm.nslm_sample_params(**{name: A + 4})) == nslm.NSLM_ERR_ALIGN, name
    assert nslm.nslm_last_launch_count() == 0
