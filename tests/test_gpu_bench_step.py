"""The benchmark's step computes what it says (needs a B200): the GEMVs and GEMMs
of its layer sets, run in the step's order on its one workspace, against fp32
products of the dequantized weights."""
import pytest
import torch

import bench
import weight_only_quantization_wise_b200 as qz

pytestmark = pytest.mark.gpu


def test_products_of_a_step():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    ls = bench.LayerSet(qz, torch.device("cuda:0"))
    outs = ls.y4 + ls.y8 + ls.yg + ls.y4_70 + ls.y8_70
    for _ in range(3):
        for y in outs:
            y.zero_()
        for part in (ls.gemv4, ls.gemv8, ls.gemv4_70b, ls.gemv8_70b, ls.gemm):
            part(0)
    assert qz.qz_device_status() == 0
    # bf16's half step, 2^-8 of the value; K / 16 tensor core sums of 16 products in a
    # chain and at most 64 joins, each off by at most 2^-22 of the largest magnitude
    # in it, which the sum of the products' magnitudes bounds
    def check(y, a, w):
        a, w = a.double(), w.double()
        want, size = a @ w.t(), a.abs() @ w.abs().t()
        lim = 2.0 ** -8 * want.abs() + (a.shape[1] / 16 + 64) * 2.0 ** -22 * size
        assert float(((y.double() - want).abs() / lim).max()) <= 1.0

    for li, (N, K) in enumerate(bench.LAYERS):
        w4 = qz.qz_dequantize(ls.c4[0][li], ls.s4[0][li], ls.z4[0][li], N, K, 4, False, bench.GROUP)
        w8 = qz.qz_dequantize(ls.c8[0][li], ls.s8[0][li], None, N, K, 8, True, K)
        check(ls.y4[li], ls.a1[li], w4)
        check(ls.y8[li], ls.a1[li], w8)
        check(ls.yg[li], ls.ap[li], w4)
    for li, (N, K) in enumerate(bench.LAYERS_70B):
        w4 = qz.qz_dequantize(ls.c4_70[li][0], ls.s4_70[li][0], ls.z4_70[li][0], N, K, 4, False,
                              bench.GROUP)
        w8 = qz.qz_dequantize(ls.c8_70[li][0], ls.s8_70[li][0], None, N, K, 8, True, K)
        check(ls.y4_70[li], ls.a1_70[li], w4)
        check(ls.y8_70[li], ls.a1_70[li], w8)
