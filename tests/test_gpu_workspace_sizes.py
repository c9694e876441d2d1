"""Bytes a Workspace holds, and one buffer under calls of every size (needs a
B200): split-K counters stand in the last QZ_WORKSPACE_COUNTERS bytes of a
buffer that has them to spare, where no call's partial sums reach."""
import random

import pytest
import torch

import synthetic
import weight_only_quantization_wise_b200 as qz

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


class Layer:
    """A packed layer's calls of any M; each takes (M, workspace, out)."""

    def __init__(self, dev, N, K, seed):
        self.N, self.K = N, K
        w = synthetic.weights(N, K, seed=seed, device=dev)
        self.p4 = qz.qz_quantize_pack(w, 4, False, 128)
        self.p8 = qz.qz_quantize_pack(w, 8, True, K)[:2]
        self.pf = qz.qz_fp4_quantize(w, qz.QZ_FP4_MX)
        self.acts = synthetic.activations(600, K, seed=seed, device=dev)
        g = torch.Generator().manual_seed(seed)
        self.adapters = (torch.randn(3, 16, K, generator=g).to(torch.bfloat16).to(dev),
                         torch.randn(3, N, 16, generator=g).to(torch.bfloat16).to(dev),
                         torch.randint(-1, 3, (64,), generator=g, dtype=torch.int32).to(dev),
                         torch.ones(3, device=dev))

    def lora(self, M):
        down, up, ids, ls = self.adapters
        return down, up, ids[:M], ls

    def ops(self, M):
        N, K, a = self.N, self.K, self.acts[:M]
        if M > 64:
            return [(qz.QZ_OP_W4A16_GEMM, 128, lambda ws: qz.qz_w4a16_gemm(a, *self.p4, N, K, 128, workspace=ws)),
                    (qz.QZ_OP_W8A16_GEMM, K, lambda ws: qz.qz_w8a16_gemm(a, *self.p8, N, K, workspace=ws))]
        out = [(qz.QZ_OP_W4A16_GEMV, 128, lambda ws: qz.qz_w4a16_gemv(a, *self.p4, N, K, 128, workspace=ws)),
               (qz.QZ_OP_W8A16_GEMV, K, lambda ws: qz.qz_w8a16_gemv(a, *self.p8, N, K, workspace=ws)),
               (qz.QZ_OP_W4A16_LORA_GEMV, 128, lambda ws: qz.qz_w4a16_lora_gemv(
                   a, *self.p4, N, K, *self.lora(M), workspace=ws)),
               (qz.QZ_OP_W8A16_LORA_GEMV, K, lambda ws: qz.qz_w8a16_lora_gemv(
                   a, *self.p8, N, K, *self.lora(M), workspace=ws))]
        if M <= 16:
            out.append((qz.QZ_OP_FP4A16_GEMV, 0, lambda ws: qz.qz_fp4a16_gemv(
                a, *self.pf, N, K, qz.QZ_FP4_MX, workspace=ws)))
        return out


@pytest.fixture(scope="module")
def layers(dev):
    # the last one has more 128-row tasks than CTAs, each of two K blocks
    return [Layer(dev, 4096, 4096, 1), Layer(dev, 1024, 8192, 2), Layer(dev, 300, 2048, 3),
            Layer(dev, 64100, 512, 4)]


def calls(layers, seed, n):
    rng = random.Random(seed)
    out = []
    for _ in range(n):
        layer = rng.choice(layers)
        M = rng.choice([1, 1, 2, rng.randint(1, 16), rng.randint(17, 64), rng.randint(65, 600)])
        op, g, f = rng.choice(layer.ops(M))
        out.append((f, qz.qz_workspace_bytes(op, M, layer.N, layer.K, g)))
    return out


def test_a_workspace_holds_what_its_largest_call_needs(dev, layers):
    """Calls of many lengths and shapes through one Workspace: the results of
    calls of their own, and no more memory than the largest call's (a buffer of
    every length would come to hundreds of MB)."""
    todo = calls(layers, 1, 120)
    want = [f(None) for f, _ in todo]
    torch.cuda.synchronize()
    ws, base = qz.Workspace(dev), torch.cuda.memory_allocated(dev)
    for _ in range(2):
        for (f, _), y in zip(todo, want):
            assert torch.equal(f(ws), y)
    torch.cuda.synchronize()
    most = max(n for _, n in todo)
    # the caching allocator hands out whole pieces of 512 bytes
    assert torch.cuda.memory_allocated(dev) - base <= most + qz.QZ_WORKSPACE_COUNTERS + 1024
    assert qz.qz_device_status() == 0


@pytest.mark.parametrize("overlap", [0, 1])
def test_a_tensor_with_room_for_the_counters_serves_every_size(dev, layers, overlap):
    todo = calls(layers, 2, 60)
    want = [f(None) for f, _ in todo]
    own = torch.zeros(max(n for _, n in todo) + qz.QZ_WORKSPACE_COUNTERS, dtype=torch.uint8,
                      device=dev)
    torch.cuda.synchronize()
    qz.qz_set_launch_overlap(overlap)
    try:
        for _ in range(2):
            got = [f(own) for f, _ in todo]
            assert all(torch.equal(x, y) for x, y in zip(got, want))
            assert int(own[-qz.QZ_WORKSPACE_COUNTERS:].count_nonzero()) == 0
    finally:
        qz.qz_set_launch_overlap(0)
    assert qz.qz_device_status() == 0


def test_quantizer_and_gptq_keep_out_of_the_shared_buffer(dev, layers):
    """The per-tensor quantizer's word and GPTQ's matrices beside split-K calls."""
    ws = qz.Workspace(dev)
    w = synthetic.weights(128, 256, seed=5, device=dev)
    x = synthetic.activations(64, 256, seed=5, device=dev)
    steps = [lambda k: layers[1].ops(4)[0][2](k),
             lambda k: qz.qz_quantize_pack(w, 8, True, 0, workspace=k)[1],
             lambda k: qz.qz_gptq_quantize(w, x, 4, False, 128, workspace=k)[0],
             lambda k: layers[0].ops(8)[1][2](k)]
    want = [f(None) for f in steps]
    for _ in range(3):
        for f, y in zip(steps, want):
            assert torch.equal(f(ws), y)


def test_a_graph_keeps_its_buffer_when_the_workspace_grows(dev, layers):
    """A graph captured on a small buffer, replayed after a larger call has made
    the Workspace take another and the memory has been handed out again."""
    small, large = layers[2].ops(4)[0][2], layers[0].ops(48)[0][2]
    ws = qz.Workspace(dev)
    want = small(ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = small(ws)
    large(ws)
    torch.cuda.synchronize()
    filled = [torch.full((n,), 0x55, dtype=torch.uint8, device=dev)
              for n in (1 << 10, 1 << 14, 1 << 16, 1 << 18, 1 << 20) for _ in range(8)]
    for _ in range(3):
        y.zero_()
        graph.replay()
        assert torch.equal(y, want)
    assert all(bool((t == 0x55).all()) for t in filled)


def test_a_capture_does_not_leave_an_unfilled_buffer_behind(dev, layers):
    """The first calls of a Workspace inside a capture, then calls outside it
    before the graph has ever run, then the graph."""
    f, g = layers[1].ops(3)[0][2], layers[0].ops(2)[1][2]
    want = f(None), g(None)
    ws = qz.Workspace(dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, z = f(ws), g(ws)
    for _ in range(2):
        assert torch.equal(f(ws), want[0]) and torch.equal(g(ws), want[1])
        y.zero_(), z.zero_()
        graph.replay()
        assert torch.equal(y, want[0]) and torch.equal(z, want[1])
