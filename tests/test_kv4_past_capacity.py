"""Lengths beyond what a page table holds: the positions behind it have no keys,
and the queries keep their own positions."""
import ctypes

import numpy as np
import pytest
import torch

import kv4_ref as ref
import weight_only_quantization_wise_b200 as qz
from test_kv4_index import ix  # noqa: F401  (a fixture)


@pytest.mark.parametrize("window", [0, 1, 5, 16, 40, 1000])
@pytest.mark.parametrize("L", [64, 65, 70, 80, 200, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [1, 10, 70])
def test_units_cover_every_key_that_a_row_sees(ix, L, n, window):  # noqa: F811
    capacity, o = 64, (ctypes.c_longlong * 6)()
    ix.s_seq_work(3, 3 + n, L, 100, capacity, window, 2, 4, 8, o)
    assert o[0] == n and o[1] == 64 and o[3] >= 1 and o[5] == o[4] * 4 * o[3]
    assert 0 <= o[2] and (o[2] + o[3]) * 16 <= capacity + 16
    for i in range(n):
        p = L - n + i
        lo, hi = max(0, p - window + 1 if window else 0), min(p, capacity - 1)
        if p >= 0 and lo <= hi:
            assert o[2] * 16 <= lo and hi < (o[2] + o[3]) * 16


@pytest.mark.gpu
@pytest.mark.parametrize("D,g", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("window", [0, 12, 20])
@pytest.mark.parametrize("L", [70, 2 ** 31 - 1])
def test_queries_keep_their_positions(D, g, window, L):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from test_gpu_kv4 import Cache, i32, keys, randn
    dev, H, new, cap = torch.device("cuda:0"), 2, 10, 64
    k, v = keys((cap, H, D), 91), randn((cap, H, D), 92)
    c = Cache(dev, [cap], H, D, 16, g)
    c.append(k.to(dev), v.to(dev), [cap], [cap])
    c.table = c.table[:, :cap // 16].contiguous()
    q = randn((new, 2 * H, D), 93)
    got = qz.qz_kv4_attention(q.to(dev), c.buf, c.table, i32([L], dev), i32([0, new], dev), H, 16, g,
                              window=window).cpu().double().numpy()
    assert qz.qz_device_status() == qz.QZ_ERR_DEVICE_INDEX
    L = min(L, cap + new + window)                   # all rows beyond the last window alike
    kq, vq = ref.quantize(k, g), ref.quantize(v, g)
    kv = [ref.values(*kq, g), ref.values(*vq, g), ref.bf16_f64(kq[1]).max(-1),
          ref.bf16_f64(vq[1]).max(-1)]
    kv = tuple(np.concatenate([x, np.zeros((L - cap,) + x.shape[1:])]) for x in kv)
    want, parts = ref.attention(q.double().numpy(), [kv], [L], [new], D ** -0.5, window,
                                [np.arange(L) >= cap])
    assert (np.abs(got - want) <= ref.bound(want, parts, D)).all()
