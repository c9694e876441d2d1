"""Host-side refusals of the LoRA GEMVs (no GPU: fake addresses that are never
dereferenced; every call is rejected by the checks before any launch)."""
import ctypes

import pytest

import weight_only_quantization_wise_b200 as qz

INVALID, ALIGN, UNSUP, WS = 1, 2, 3, 4
P = [ctypes.c_void_p(0x10000 * i) for i in range(1, 12)]
MIS = ctypes.c_void_p(0x10008)
BIG = 1 << 40

GOOD = dict(a=P[0], codes=P[1], scales=P[2], zeros=P[3], M=4, N=256, K=512, g=128, la=P[4],
            lb=P[5], ids=P[6], ls=P[7], n=3, rank=16, y=P[8], ws=P[9], wb=BIG)


def w4(**kw):
    v = dict(GOOD, **kw)
    return qz.lib.qz_w4a16_lora_gemv(*(v[k] for k in (
        "a", "codes", "scales", "zeros", "M", "N", "K", "g", "la", "lb", "ids", "ls", "n", "rank",
        "y", "ws", "wb")), None)


def w8(**kw):
    v = dict(GOOD, **kw)
    return qz.lib.qz_w8a16_lora_gemv(*(v[k] for k in (
        "a", "codes", "scales", "M", "N", "K", "la", "lb", "ids", "ls", "n", "rank", "y", "ws",
        "wb")), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(M=0), INVALID), (dict(M=65), UNSUP), (dict(K=192), UNSUP), (dict(N=0), INVALID),
    (dict(a=None), INVALID), (dict(codes=MIS), ALIGN), (dict(y=None), INVALID),
    (dict(la=None), INVALID), (dict(lb=None), INVALID), (dict(ids=None), INVALID),
    (dict(ls=None), INVALID), (dict(la=MIS), ALIGN), (dict(lb=MIS), ALIGN),
    (dict(ids=ctypes.c_void_p(0x10002)), ALIGN), (dict(ls=ctypes.c_void_p(0x10002)), ALIGN),
    (dict(n=0), INVALID), (dict(n=1 << 31), INVALID), (dict(n=(1 << 31) - 1, rank=128, N=1 << 20), INVALID),
    (dict(rank=0), INVALID), (dict(rank=12), UNSUP), (dict(rank=136), UNSUP),
    (dict(ws=None), WS), (dict(wb=100), WS), (dict(ws=MIS), ALIGN),
])
def test_refusals(kw, expect):
    assert w4(**kw) == expect
    assert w8(**kw) == expect


@pytest.mark.parametrize("kw,expect", [(dict(g=0), INVALID), (dict(g=48), INVALID),
                                       (dict(g=16), UNSUP), (dict(zeros=None), INVALID)])
def test_w4_refusals(kw, expect):
    assert w4(**kw) == expect


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (64, 130, 512), (16, 28672, 8192)])
def test_workspace(M, N, K):
    """Two bf16 halves of M x 128 products, then the plain GEMV's workspace."""
    for op, base, g in ((qz.QZ_OP_W4A16_LORA_GEMV, qz.QZ_OP_W4A16_GEMV, 128),
                        (qz.QZ_OP_W8A16_LORA_GEMV, qz.QZ_OP_W8A16_GEMV, K)):
        assert (qz.qz_workspace_bytes(op, M, N, K, g) ==
                M * 128 * 4 + qz.qz_workspace_bytes(base, M, N, K, g))
    with pytest.raises(qz.QzError):
        qz.qz_workspace_bytes(qz.QZ_OP_W4A16_LORA_GEMV, 65, N, K, 128)
