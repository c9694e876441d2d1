"""What the 4-bit cache holds does not depend on how a prompt was cut into calls
(needs a B200): tokens stored one or two at a time, and many at once, values that
are not finite among them."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import weight_only_quantization_wise_b200 as qz
from test_gpu_kv4 import Cache, dev, edge_rows, randn  # noqa: F401  (dev is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("cuts", [[1] * 40, [2] * 20, [1, 3, 12, 2, 14, 1, 7], [17, 2, 21]])
def test_cuts_of_a_prompt(dev, D, g, cuts):  # noqa: F811
    H, L = 2, 40
    k, v = edge_rows(L, H, D, 81), randn((L, H, D), 82)
    inf, nan = float("inf"), float("nan")
    for x in (k, v):
        for t, (d, value) in enumerate([(0, nan), (5, inf), (6, -inf), (D - 1, nan), (9, 3e38)]):
            x[6 + 5 * t, 0, d] = value
        x[7, 1, :2] = torch.tensor([inf, -inf])
        x[8, 1, :3] = torch.tensor([inf, nan, -1.0])
        x[9, 1, :2] = torch.tensor([3e38, -3e38])
        x[10, 1, :g] = nan
        x[11, 1, 1:] *= 1e-38                    # a NaN beside a subnormal scale
        x[11, 1, 0] = nan
    whole, parts = (Cache(dev, [L], H, D, 32, g, fill=0x5A) for _ in range(2))
    k, v = k.to(dev), v.to(dev)
    whole.append(k, v, [L], [L])
    at = 0
    for n in cuts:
        parts.append(k[at:at + n], v[at:at + n], [at + n], [n])
        at += n
    assert at == L
    assert torch.equal(whole.buf, parts.buf)
    # the codes, scales and zeros of qz_quantize_pack
    host = whole.buf.cpu().numpy()
    for which, x in ((0, k), (1, v)):
        c, s, z = (t.cpu() for t in qz.qz_quantize_pack(x.reshape(L * H, D), 4, False, g))
        codes = torch.stack([c & 15, c >> 4], -1).reshape(L, H, D).numpy()
        s = s.view(torch.int16).reshape(L, H, D // g).numpy().view(np.uint16)
        z = z.reshape(L, H, D // g).numpy()
        for h in range(H):
            for block in range(-(-L // 16)):
                got = ref.unpack_record(whole.record(host, 0, h, block), D, g)
                n = min(16, L - 16 * block)
                for mine, want in zip(got, (codes, s, z)):
                    assert np.array_equal(mine[which, :n], want[16 * block:16 * block + n, h])
    assert qz.qz_device_status() == 0
