"""Adapter GEMVs between plain ones, each call's result the next one's input, with
launch overlap off and on, eager and captured (needs a B200)."""
import pytest
import torch

import synthetic
import weight_only_quantization_wise_b200 as qz

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 5, 16, 40])
def test_chain_with_launch_overlap(M):
    """A decode step's order: an overlapped GEMV may start before the adapter GEMV
    in front of it ends, and an adapter GEMV before a plain one ends."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev, N, g, R, n = torch.device("cuda:0"), 2048, 128, 32, 4
    gen = torch.Generator().manual_seed(M)
    ws = qz.Workspace(dev)
    layers = []
    for i in range(8):
        w = synthetic.weights(N, N, seed=i, device=dev)
        down = (torch.randn(n, R, N, generator=gen) * N ** -0.5).to(torch.bfloat16).to(dev)
        up = (torch.randn(n, N, R, generator=gen) * 0.1).to(torch.bfloat16).to(dev)
        ids = torch.randint(-1, n, (M,), generator=gen, dtype=torch.int32).to(dev)
        ls = torch.rand(n, generator=gen).to(dev)
        if i % 4 < 2:
            c, s, z = qz.qz_quantize_pack(w, 4, False, g)
            plain = lambda a, y, c=c, s=s, z=z: qz.qz_w4a16_gemv(a, c, s, z, N, N, g, y=y, workspace=ws)  # noqa: E731
            lora = lambda a, y, c=c, s=s, z=z, x=(down, up, ids, ls): qz.qz_w4a16_lora_gemv(  # noqa: E731
                a, c, s, z, N, N, *x, group_size=g, y=y, workspace=ws)
        else:
            c, s, _ = qz.qz_quantize_pack(w, 8, True, N)
            plain = lambda a, y, c=c, s=s: qz.qz_w8a16_gemv(a, c, s, N, N, y=y, workspace=ws)  # noqa: E731
            lora = lambda a, y, c=c, s=s, x=(down, up, ids, ls): qz.qz_w8a16_lora_gemv(  # noqa: E731
                a, c, s, N, N, *x, y=y, workspace=ws)
        layers.append(lora if i % 2 else plain)
    x0 = synthetic.activations(M, N, seed=3, device=dev)
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device=dev) for _ in layers]

    def step(sync=False):
        a = x0
        for f, y in zip(layers, outs):
            f(a, y)
            if sync:
                torch.cuda.synchronize()
            a = y

    step(sync=True)
    want = [y.clone() for y in outs]
    assert all(bool(y.isfinite().all()) for y in want)
    for overlap in (0, 1):
        qz.qz_set_launch_overlap(overlap)
        try:
            for _ in range(20):
                for y in outs:
                    y.zero_()
                step()
                assert all(torch.equal(y, t) for y, t in zip(outs, want))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(20):
                for y in outs:
                    y.zero_()
                graph.replay()
                assert all(torch.equal(y, t) for y, t in zip(outs, want))
        finally:
            qz.qz_set_launch_overlap(0)
    assert qz.qz_device_status() == 0
