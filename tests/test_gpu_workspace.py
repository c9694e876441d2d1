"""One Workspace under calls of different sizes (needs a B200): where a split-K
call keeps its arrival counters depends on its sizes, so another call's partial
sums must not lie over them."""
import pytest
import torch

import synthetic
import weight_only_quantization_wise_b200 as qz

pytestmark = pytest.mark.gpu


def test_one_workspace_serves_calls_of_different_sizes():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    ws = qz.Workspace(dev)
    layers = []
    for i, (N, K, M) in enumerate([(4096, 4096, 1), (1024, 8192, 16), (4096, 4096, 4), (300, 2048, 8)]):
        w = synthetic.weights(N, K, seed=i, device=dev)
        a = synthetic.activations(M, K, seed=i, device=dev)
        c, s, z = qz.qz_quantize_pack(w, 4, False, 128)
        c8, s8, _ = qz.qz_quantize_pack(w, 8, True, K)
        sm = torch.empty(s.numel() + 1, dtype=s.dtype, device=dev)[1:].view(s.shape)
        sm.copy_(s)                                 # scales that are not 16-byte aligned
        layers += [lambda w_, a=a, c=c, s=s, z=z, N=N, K=K: qz.qz_w4a16_gemv(
                       a, c, s, z, N, K, 128, workspace=w_),
                   lambda w_, a=a, c=c, s=sm, z=z, N=N, K=K: qz.qz_w4a16_gemv(
                       a, c, s, z, N, K, 128, workspace=w_),
                   lambda w_, a=a, c=c8, s=s8, N=N, K=K: qz.qz_w8a16_gemv(
                       a, c, s, N, K, workspace=w_)]
    want = [f(None) for f in layers]
    for _ in range(3):
        for f, y in zip(layers, want):
            assert torch.equal(f(ws), y)
