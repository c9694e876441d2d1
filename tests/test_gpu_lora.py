"""Low-rank adapters beside packed projections on the GPU (needs a B200): against
the fp64 product over the oracle's dequantized weights plus the adapters in fp64,
and a decode step of projections, cache and attention together."""
import numpy as np
import pytest
import torch

import kv4_ref as ref
import oracle
import synthetic
import weight_only_quantization_wise_b200 as qz

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def randn(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def adapter_set(n, N, K, R, seed):
    g = torch.Generator().manual_seed(seed + 5)
    return (randn((n, R, K), seed, K ** -0.5), randn((n, N, R), seed + 1, 0.1),
            torch.rand(n, generator=g) * 2 - 0.5)


def reference(w, a, down, up, ids, ls, bits, g):
    """float64 result and the bound's magnitude terms."""
    N, K = w.shape
    sym, gs = (False, g) if bits == 4 else (True, K)
    c, s, z = oracle.quantize_pack(synthetic.bf16_bits(w), bits, sym, gs)
    w_hat = oracle.dequantize(c, s, z, N, K, bits, sym, gs)
    y, mag = oracle.matmul_f64(synthetic.bf16_bits(a), w_hat)
    low, lmag = np.zeros_like(y), np.zeros_like(y)
    d, u, x = (t.double().numpy() for t in (down, up, a))
    for m, r in enumerate(ids):
        if 0 <= r < len(ls):
            low[m] = float(ls[r]) * (u[r] @ (d[r] @ x[m]))
            lmag[m] = abs(float(ls[r])) * (np.abs(u[r]) @ (np.abs(d[r]) @ np.abs(x[m])))
    return y + low, mag, lmag


def bound(y, mag, lmag):
    """Half a bf16 step; the projection's own term (the plain GEMV's: its fp32
    sums); the adapter's: h = hi + lo holds 2^-17, its sums run over at most 32
    products of 16 per warp (2^-22 each, 2^-17) and 16 partial sums (2^-20), the
    second product over at most 16 (2^-18): below 2^-15 of the magnitudes."""
    return 2.0 ** -8 * np.abs(y) + 1e-4 * mag + 2.0 ** -15 * lmag + 2.0 ** -133


def run(dev, bits, w, a, down, up, ids, ls, g, ws=None, stream=None):
    N, K = w.shape
    args = [t.to(dev) for t in (down, up, torch.tensor(ids, dtype=torch.int32), ls)]
    if bits == 4:
        c, s, z = qz.qz_quantize_pack(w.to(dev), 4, False, g)
        return qz.qz_w4a16_lora_gemv(a.to(dev), c, s, z, N, K, *args, group_size=g, workspace=ws,
                                     stream=stream)
    c, s, _ = qz.qz_quantize_pack(w.to(dev), 8, True, K)
    return qz.qz_w8a16_lora_gemv(a.to(dev), c, s, N, K, *args, workspace=ws, stream=stream)


def check(dev, bits, N, K, g, M, R, n, ids, seed=0):
    w, a = synthetic.weights(N, K, seed=seed), synthetic.activations(M, K, seed=seed)
    down, up, ls = adapter_set(n, N, K, R, seed)
    y = run(dev, bits, w, a, down, up, ids, ls, g)
    torch.cuda.synchronize()
    want, mag, lmag = reference(w, a, down, up, ids, ls, bits, g)
    err = np.abs(y.cpu().double().numpy() - want)
    assert (err <= bound(want, mag, lmag)).all(), (err / bound(want, mag, lmag)).max()


def mixed_ids(M, n, seed):
    rng = np.random.default_rng(seed)
    return rng.integers(-1, n, M).tolist()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 64])
def test_tokens(dev, bits, M):
    check(dev, bits, 384, 512, 128, M, 16, 5, mixed_ids(M, 5, M), seed=M)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("R", [8, 16, 24, 32, 40, 64, 72, 128])
def test_ranks(dev, bits, R):
    check(dev, bits, 200, 384, 64, 6, R, 3, [0, 2, -1, 2, 1, 0], seed=R)


@pytest.mark.parametrize("N,K,g", [(17, 128, 32), (1, 256, 128), (300, 1024, 64), (1000, 4096, 128),
                                   (4096, 11008, 128), (130, 5632, 256)])
@pytest.mark.parametrize("M", [1, 5, 20])
def test_shapes(dev, N, K, g, M):
    check(dev, 4, N, K, g, M, 16, 4, mixed_ids(M, 4, N), seed=N)


def test_all_tokens_share_one_adapter(dev):
    check(dev, 4, 256, 1024, 128, 64, 32, 3, [1] * 64)


def test_every_token_its_own_adapter(dev):
    check(dev, 8, 256, 512, 512, 64, 8, 64, list(range(63, -1, -1)))


@pytest.mark.parametrize("bits", [4, 8])
def test_tokens_without_adapter_get_the_plain_projection(dev, bits):
    N, K, M = 500, 1024, 9
    w, a = synthetic.weights(N, K, seed=3), synthetic.activations(M, K, seed=3)
    down, up, ls = adapter_set(2, N, K, 16, 1)
    y = run(dev, bits, w, a, down, up, [-1] * M, ls, 128)
    if bits == 4:
        c, s, z = qz.qz_quantize_pack(w.to(dev), 4, False, 128)
        plain = qz.qz_w4a16_gemv(a.to(dev), c, s, z, N, K, 128)
    else:
        c, s, _ = qz.qz_quantize_pack(w.to(dev), 8, True, K)
        plain = qz.qz_w8a16_gemv(a.to(dev), c, s, N, K)
    assert torch.equal(y, plain)


def test_unused_adapters_are_not_read_and_wild_indices_are_reported(dev):
    N, K = 256, 512
    w, a = synthetic.weights(N, K, seed=4), synthetic.activations(4, K, seed=4)
    down, up, ls = adapter_set(3, N, K, 16, 2)
    down[1], up[1], ls[1] = float("nan"), float("inf"), float("nan")
    assert qz.qz_device_status() == 0
    y = run(dev, 4, w, a, down, up, [0, -2 ** 31, 3, 2], ls, 128)
    assert qz.qz_device_status() == qz.QZ_ERR_DEVICE_INDEX and qz.qz_device_status() == 0
    want, mag, lmag = reference(w, a, down, up, [0, -1, -1, 2], ls, 4, 128)
    err = np.abs(y.cpu().double().numpy() - want)
    assert (err <= bound(want, mag, lmag)).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("M", [4, 12, 40])
@pytest.mark.parametrize("where", ["down", "up", "scale"])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_an_adapter_that_is_not_finite_harms_its_own_tokens_alone(dev, bits, M, where, value):
    N, K, R = 200, 512, 24
    w, a = synthetic.weights(N, K, seed=6), synthetic.activations(M, K, seed=6)
    down, up, ls = adapter_set(3, N, K, R, 4)
    ids = [m % 4 - 1 for m in range(M)]
    clean = run(dev, bits, w, a, down, up, ids, ls, 128)
    {"down": down, "up": up, "scale": ls}[where][1] = value
    got = run(dev, bits, w, a, down, up, ids, ls, 128)
    others = [m for m in range(M) if ids[m] != 1]
    assert torch.equal(got[others], clean[others])
    assert not got[[m for m in range(M) if ids[m] == 1]].isfinite().any()


@pytest.mark.parametrize("bits", [4, 8])
def test_a_low_rank_product_past_bf16_is_infinite(dev, bits):
    """512 products of 1e37 pass the largest number: the output's sign is B's."""
    N, K, M = 128, 512, 2
    w, a = synthetic.weights(N, K, seed=7), torch.ones(M, K, dtype=torch.bfloat16)
    down, up = torch.full((1, 8, K), 1e37), torch.ones(1, N, 8)
    up[0, N // 2:] = -1.0
    y = run(dev, bits, w, a, down.to(torch.bfloat16), up.to(torch.bfloat16), [0] * M,
            torch.ones(1), 128)
    assert (y[:, :N // 2] == float("inf")).all() and (y[:, N // 2:] == float("-inf")).all()


def test_adapter_gradients_of_scale(dev):
    """y is affine in lora_scales: the difference of two calls is the adapter's
    part alone, to the rounding of the outputs."""
    N, K, M = 300, 512, 3
    w, a = synthetic.weights(N, K, seed=5), synthetic.activations(M, K, seed=5)
    down, up, ls = adapter_set(2, N, K, 32, 3)
    ids = [0, 1, 0]
    y1 = run(dev, 4, w, a, down, up, ids, ls, 128).cpu().double().numpy()
    y0 = run(dev, 4, w, a, down, up, ids, torch.zeros(2), 128).cpu().double().numpy()
    w1, m1, l1 = reference(w, a, down, up, ids, ls, 4, 128)
    w0, m0, l0 = reference(w, a, down, up, ids, torch.zeros(2), 4, 128)
    assert (np.abs((y1 - y0) - (w1 - w0)) <= bound(w1, m1, l1) + bound(w0, m0, l0)).all()


def test_repeatable_with_a_shared_workspace_and_in_a_graph(dev):
    N, K, M, g = 1024, 4096, 12, 128
    w, a = synthetic.weights(N, K, seed=6), synthetic.activations(M, K, seed=6)
    down, up, ls = adapter_set(4, N, K, 64, 4)
    c, s, z = qz.qz_quantize_pack(w.to(dev), 4, False, g)
    ids = torch.tensor(mixed_ids(M, 4, 1), dtype=torch.int32, device=dev)
    down, up, ls, a = (t.to(dev) for t in (down, up, ls, a))
    ws = qz.Workspace(dev)
    call = lambda y=None: qz.qz_w4a16_lora_gemv(a, c, s, z, N, K, down, up, ids, ls, workspace=ws, y=y)  # noqa: E731
    first = call()
    for _ in range(10):
        assert torch.equal(call(), first)
        qz.qz_w4a16_gemv(a, c, s, z, N, K, g, workspace=ws)
    out = torch.zeros_like(first)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        call(out)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
        call(out)
    for i in range(3):
        new = synthetic.activations(M, K, seed=20 + i).to(dev)
        a.copy_(new)
        ids.copy_(torch.tensor(mixed_ids(M, 4, 7 + i), dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call())
    st = torch.cuda.Stream(dev)
    torch.cuda.synchronize()
    y = qz.qz_w4a16_lora_gemv(a, c, s, z, N, K, down, up, ids, ls, stream=st)
    st.synchronize()
    assert torch.equal(y, out)


def test_python_argument_checks(dev):
    N, K = 64, 128
    w, a = synthetic.weights(N, K, seed=1).to(dev), synthetic.activations(2, K, seed=1).to(dev)
    c, s, z = qz.qz_quantize_pack(w, 4, False, 128)
    down, up, ls = (t.to(dev) for t in adapter_set(2, N, K, 16, 0))
    ids = torch.zeros(2, dtype=torch.int32, device=dev)
    good = dict(lora_a=down, lora_b=up, adapters=ids, lora_scales=ls)
    for bad in (dict(lora_a=down.float()), dict(lora_a=down[:, :, :64]), dict(lora_b=up[:1]),
                dict(adapters=ids.long()), dict(adapters=ids[:1]), dict(lora_scales=ls.double()),
                dict(lora_scales=ls.cpu()), dict(lora_b=up.transpose(0, 1).contiguous())):
        with pytest.raises(ValueError):
            qz.qz_w4a16_lora_gemv(a, c, s, z, N, K, **dict(good, **bad))
    for bad in ((c[:, :32], s, z), (c, s.float(), z), (c, s, z[:1]), (c.cpu(), s, z)):
        with pytest.raises(ValueError):
            qz.qz_w4a16_lora_gemv(a, *bad, N, K, down, up, ids, ls)
    with pytest.raises(ValueError):
        qz.qz_w4a16_lora_gemv(a, c, s, z, N, K, down, up, ids, ls, y=torch.empty_like(a))
    with pytest.raises(qz.QzError):                  # rank not a multiple of 8
        qz.qz_w4a16_lora_gemv(a, c, s, z, N, K, down[:, :12].contiguous(),
                              up[:, :, :12].contiguous(), ids, ls)


@pytest.mark.parametrize("normed", [False, True])
def test_decode_step_of_a_layer(dev, normed):
    """Query, key and value projections with adapters, the cache, attention, and
    the output projection, step after step, against the same chain in float64
    that takes each stage's own inputs.  Without a norm the activations grow until
    every softmax picks one key."""
    H, share, D, g, page, K, R, B = 2, 4, 64, 64, 16, 512, 16, 3
    heads = H * share
    N = (heads + 2 * H) * D
    wq, wo = synthetic.weights(N, K, 0.05, 1), synthetic.weights(K, heads * D, 0.05, 2)
    packed = [qz.qz_quantize_pack(w.to(dev), 4, False, 128) for w in (wq, wo)]
    ads = [adapter_set(2, N, K, R, 3), adapter_set(2, K, heads * D, R, 4)]
    dads = [tuple(t.to(dev) for t in x) for x in ads]
    ids = [1, -1, 0]
    dids = torch.tensor(ids, dtype=torch.int32, device=dev)
    steps, lens = 20, [0, 0, 0]
    table = torch.arange(B * 2, dtype=torch.int32, device=dev).view(B, 2)
    cache = torch.zeros(qz.qz_kv4_cache_bytes(B * 2, H, D, page, g), dtype=torch.uint8, device=dev)
    cu = torch.arange(B + 1, dtype=torch.int32, device=dev)
    kv_lens = torch.zeros(B, dtype=torch.int32, device=dev)
    ws = qz.Workspace(dev)
    x = synthetic.activations(B, K, seed=9)
    ks = [torch.zeros((0, H, D), dtype=torch.bfloat16) for _ in range(B)]
    vs = [torch.zeros((0, H, D), dtype=torch.bfloat16) for _ in range(B)]
    for _ in range(steps):
        kv_lens.add_(1)
        qkv = qz.qz_w4a16_lora_gemv(x.to(dev), *packed[0], N, K, dads[0][0], dads[0][1], dids,
                                    dads[0][2], workspace=ws).view(B, heads + 2 * H, D)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + H], qkv[:, heads + H:]
        qz.qz_kv4_append(cache, k, v, table, kv_lens, cu, page, g)
        o = qz.qz_kv4_attention(q, cache, table, kv_lens, cu, H, page, g, workspace=ws)
        y = qz.qz_w4a16_lora_gemv(o.view(B, heads * D), *packed[1], K, heads * D, dads[1][0],
                                  dads[1][1], dids, dads[1][2], workspace=ws)
        want, mag, lmag = reference(wq, x, *ads[0][:2], ids, ads[0][2], 4, 128)
        assert (np.abs(qkv.cpu().double().numpy().reshape(B, N) - want) <= bound(want, mag, lmag)).all()
        lens = [n + 1 for n in lens]
        kv = []
        for b in range(B):
            ks[b] = torch.cat([ks[b], k[b:b + 1].cpu()])
            vs[b] = torch.cat([vs[b], v[b:b + 1].cpu()])
            kq, vq = ref.quantize(ks[b], g), ref.quantize(vs[b], g)
            kv.append((ref.values(*kq, g), ref.values(*vq, g), ref.bf16_f64(kq[1]).max(-1),
                       ref.bf16_f64(vq[1]).max(-1)))
        att, parts = ref.attention(q.cpu().double().numpy(), kv, lens, [1] * B, D ** -0.5, 0)
        assert (np.abs(o.cpu().double().numpy() - att) <= ref.bound(att, parts, D)).all()
        oc = o.cpu().reshape(B, heads * D)
        want, mag, lmag = reference(wo, oc, *ads[1][:2], ids, ads[1][2], 4, 128)
        assert (np.abs(y.cpu().double().numpy() - want) <= bound(want, mag, lmag)).all()
        x = y.cpu().float() + x.float()
        if normed:
            x = x / x.square().mean(-1, keepdim=True).sqrt()
        x = x.to(torch.bfloat16)
    assert qz.qz_device_status() == 0
