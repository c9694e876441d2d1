"""The paged 4-bit key/value cache on the GPU (needs a B200): append against the
CPU oracle's quantize_pack byte for byte, read against its dequantize, attention
against a plain 64-bit form within kv4_ref.bound."""
import random

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


def keys(shape, seed):
    g = torch.Generator().manual_seed(seed)
    gain = 1 + 7 * (torch.rand(shape[1:], generator=g) < 0.05)
    return (torch.randn(shape, generator=g) * gain + torch.randn(shape[1:], generator=g)).to(
        torch.bfloat16)


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Cache:
    """A cache with scattered pages, filled with garbage (NaN scales) first."""

    def __init__(self, dev, lens, H, D, page, g, seed=0, spare=2, fill=0xFF):
        self.dev, self.H, self.D, self.page, self.g = dev, H, D, page, g
        need = [-(-n // page) for n in lens]
        self.pages = sum(need) + spare
        order = list(range(self.pages))
        random.Random(seed).shuffle(order)
        self.rows, at = [], 0
        width = max(1, max(need)) + 1
        for n in need:
            self.rows.append(order[at:at + n] + [-7] * (width - n))
            at += n
        self.table = i32(self.rows, dev)
        self.buf = torch.full((qz.qz_kv4_cache_bytes(self.pages, H, D, page, g),), fill,
                              dtype=torch.uint8, device=dev)

    def append(self, k, v, lens, new, **kw):
        qz.qz_kv4_append(self.buf, k, v, self.table, i32(lens, self.dev),
                         i32(np.cumsum([0] + list(new)).tolist(), self.dev), self.page, self.g, **kw)

    def attend(self, q, lens, new, **kw):
        return qz.qz_kv4_attention(q, self.buf, self.table, i32(lens, self.dev),
                                   i32(np.cumsum([0] + list(new)).tolist(), self.dev), self.H,
                                   self.page, self.g, **kw)

    def read(self, lens, new, **kw):
        return qz.qz_kv4_read(self.buf, self.table, i32(lens, self.dev),
                              i32(np.cumsum([0] + list(new)).tolist(), self.dev), sum(new), self.H,
                              self.D, self.page, self.g, **kw)

    def record(self, host, b, h, block):
        pb = self.page // 16
        r = (self.rows[b][block // pb] * self.H + h) * pb + block % pb
        n = ref.record_size(self.D, self.g)
        return host[r * n:(r + 1) * n]


def edge_rows(T, H, D, seed):
    x = keys((T, H, D), seed).float()
    x[0] = 0.0
    if T > 5:
        x[1] = 3.25                                 # one value, above zero
        x[2] = -1.5
        x[3] = torch.arange(D) % 16 - 1.5           # ties at the top of the range
        x[4] = x[4] * 1e-38                         # subnormal scales
        x[5] = x[5] * 1e30
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("page", [16, 48])
def test_append_is_bit_exact(dev, D, g, page):
    """Codes, scales and zeros of every appended token are the oracle's, at the
    documented places; every other byte of the cache keeps its value; rows
    behind the last sequence change nothing."""
    H, lens, new = 3, [19, 5, 40, 1, 33], [19, 0, 7, 1, 18]
    T = sum(new)
    k, v = edge_rows(T + 3, H, D, 1), randn((T + 3, H, D), 2, 0.5)
    c = Cache(dev, lens, H, D, page, g, fill=0xA5)
    c.append(k.to(dev), v.to(dev), lens, new)
    assert qz.qz_device_status() == 0
    host = c.buf.cpu().numpy()
    want = np.full_like(host, 0xA5)
    row = 0
    kq, vq = ref.quantize(k, g), ref.quantize(v, g)
    ng = D // g
    for b, (L, n) in enumerate(zip(lens, new)):
        for i in range(n):
            pos = L - n + i
            for h in range(H):
                rec = c.record(want, b, h, pos // 16)
                t = pos % 16
                for which, (codes, s, z), place in ((0, kq, ref.k_place), (1, vq, ref.v_place)):
                    for d in range(D):
                        byte, high = place(D, t, d)
                        old = int(rec[byte])
                        code = int(codes[row, h, d])
                        rec[byte] = (old & 0x0F) | code << 4 if high else (old & 0xF0) | code
                    sc = rec[16 * D:16 * D + 64 * ng].view(np.uint16).reshape(2, ng, 16)
                    ze = rec[16 * D + 64 * ng:].reshape(2, ng, 16)
                    sc[which, :, t], ze[which, :, t] = s[row, h], z[row, h]
            row += 1
    assert np.array_equal(host, want)


@pytest.mark.parametrize("D,g", ref.COMBOS)
def test_read_is_bit_exact(dev, D, g):
    H, lens = 2, [37, 1, 0, 64]
    T = sum(lens)
    k, v = edge_rows(T, H, D, 3), randn((T, H, D), 4, 0.5)
    c = Cache(dev, lens, H, D, 32, g)
    c.append(k.to(dev), v.to(dev), lens, lens)
    new = [5, 1, 0, 64]                              # the last tokens of each
    out = [torch.full((sum(new) + 2, H, D), 7.0, dtype=torch.bfloat16, device=dev)
           for _ in range(2)]
    qz.qz_kv4_read(c.buf, c.table, i32(lens, dev), i32(np.cumsum([0] + new).tolist(), dev),
                   sum(new) + 2, H, D, 32, g, k=out[0], v=out[1])
    assert qz.qz_device_status() == 0
    starts = np.cumsum([0] + lens)
    rows = np.concatenate([np.arange(starts[b + 1] - n, starts[b + 1]) for b, n in enumerate(new)])
    for x, got in ((k, out[0]), (v, out[1])):
        cc, s, z = oracle.quantize_pack(synthetic.bf16_bits(x.reshape(T * H, D)), 4, False, g)
        w = oracle.dequantize(cc, s, z, T * H, D, 4, False, g).reshape(T, H, D)
        got = synthetic.bf16_bits(got)
        assert np.array_equal(got[:-2], w[rows])
        assert (got[-2:] == 0x40E0).all()            # rows of no sequence keep their 7.0


def check_attention(dev, D, g, page, H, share, lens, new, window=0, scale=None, seed=0, T_extra=0,
                    q_std=1.0, v_std=0.5, holes=()):
    T = sum(lens)
    k, v = keys((T, H, D), seed), randn((T, H, D), seed + 1, v_std)
    c = Cache(dev, lens, H, D, page, g, seed)
    c.append(k.to(dev), v.to(dev), lens, lens)
    assert qz.qz_device_status() == 0
    q = randn((sum(new) + T_extra, H * share, D), seed + 2, q_std)
    out = torch.full_like(q, 9.0, device=dev)
    masked = [np.zeros(n, bool) for n in lens]
    if holes:
        table = c.table.clone()
        for b, page_no, value in holes:
            table[b, page_no] = value
            masked[b][page_no * page:(page_no + 1) * page] = True
        c.table = table
    c.attend(q.to(dev), lens, new, window=window, scale=scale, out=out)
    torch.cuda.synchronize()
    assert qz.qz_device_status() == (qz.QZ_ERR_DEVICE_INDEX if holes else 0)
    scale = D ** -0.5 if scale is None else scale
    starts = np.cumsum([0] + lens)
    kq, vq = ref.quantize(k, g), ref.quantize(v, g)
    kf, vf = ref.values(*kq, g), ref.values(*vq, g)
    sk, sv = ref.bf16_f64(kq[1]).max(-1), ref.bf16_f64(vq[1]).max(-1)
    kv = [tuple(x[starts[b]:starts[b + 1]] for x in (kf, vf, sk, sv)) for b in range(len(lens))]
    want, parts = ref.attention(q.double().numpy(), kv, lens, new, scale, window, masked)
    got = out.cpu().double().numpy()
    assert np.isfinite(got).all()
    n = sum(new)
    assert (got[n:] == 9.0).all()
    err = np.abs(got[:n] - want[:n])
    lim = ref.bound(want[:n], {x: y[:n] for x, y in parts.items()}, D)
    worst = (err / lim).max() if err.size else 0.0
    assert worst <= 1.0, f"{worst} of the bound at {np.unravel_index((err / lim).argmax(), err.shape)}"
    return worst


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("H,share", [(2, 4), (1, 16), (3, 1)])
def test_attention_single_tokens(dev, D, g, H, share):
    lens = [1, 15, 16, 17, 300, 64]
    check_attention(dev, D, g, 16, H, share, lens, [1] * 6, seed=D + g + share)


@pytest.mark.parametrize("share", [1, 2, 3, 5, 7, 8, 12, 16])
@pytest.mark.parametrize("page", [16, 64, 80])
def test_attention_head_shares(dev, share, page):
    check_attention(dev, 128, 128, page, 2, share, [200, 33, 1], [1, 1, 1], seed=share)


@pytest.mark.parametrize("D,g", [(64, 32), (128, 128), (256, 64)])
@pytest.mark.parametrize("new", [[4, 4, 4], [1, 9, 30], [0, 3, 0], [17, 0, 1]])
@pytest.mark.parametrize("window", [0, 1, 20])
def test_attention_several_tokens(dev, D, g, new, window):
    check_attention(dev, D, g, 32, 2, 3, [80, 41, 33], new, window=window, seed=7)


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("lens,new,extra", [([300, 41, 90], [50, 13, 1], 0), ([300, 41, 90], [50, 12, 1], 0),
                                            ([3000], [67], 0), ([40, 0, 7], [60, 0, 2], 9)])
@pytest.mark.parametrize("window", [0, 20])
def test_attention_of_prompt_parts(dev, D, g, lens, new, extra, window):
    """Many rows per key head (64 tokens of 8 heads make 128 tiles of 8 rows,
    from where tiles of 16 are used; 63 do not), tiles cut by the sequences'
    ends, rows in front of the first key, rows of no sequence."""
    check_attention(dev, D, g, 32, 2, 8, lens, new, window=window, T_extra=extra, seed=14)


def test_attention_rows_without_keys(dev):
    """No cached tokens, and more query rows than cached tokens: the rows in
    front of the first key give zeros."""
    check_attention(dev, 128, 64, 16, 2, 4, [0, 3, 20], [2, 5, 1], seed=8)
    check_attention(dev, 64, 64, 16, 1, 1, [0, 0], [1, 1], seed=9)


def test_attention_padded_batch(dev):
    """Sequences without tokens and rows of no sequence."""
    check_attention(dev, 128, 128, 16, 2, 4, [50, 20, 7, 7], [1, 0, 1, 0], T_extra=5, seed=10)


@pytest.mark.parametrize("lens", [[2000], [5000, 3, 900], [700] * 40, [16] * 700, [3] * 1500])
def test_attention_shared_by_ctas(dev, lens):
    """Items cut by warps and CTAs, many per warp, more sequences than threads."""
    check_attention(dev, 64, 64, 16, 2, 2, lens, [1] * len(lens), seed=11)


@pytest.mark.parametrize("D,g,share", [(128, 128, 4), (128, 32, 16), (256, 128, 8)])
def test_attention_long(dev, D, g, share):
    check_attention(dev, D, g, 64, 1, share, [9001, 30], [1, 2], seed=12)


@pytest.mark.parametrize("q_std,v_std,scale", [(1e-30, 1.0, None), (30.0, 1.0, 0.5),
                                               (1.0, 1e-30, None), (1.0, 1e30, None),
                                               (1e20, 1.0, 1e-20), (1.0, 1.0, 0.0),
                                               (1.0, 1.0, -0.3)])
def test_attention_ranges(dev, q_std, v_std, scale):
    check_attention(dev, 128, 64, 16, 2, 4, [150, 40], [1, 2], q_std=q_std, v_std=v_std,
                    scale=scale, seed=13)


def test_attention_of_uneven_values(dev):
    """A key that holds nearly all the weight and has tiny values beside keys of
    little weight and large values."""
    H, D, g, L = 1, 128, 128, 40
    k, v = torch.zeros(L, H, D), torch.randn(L, H, D, generator=torch.Generator().manual_seed(1))
    k[0] = 1.0
    v[0] *= 2.0 ** -12
    q = torch.full((1, H, D), 0.8)
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    c = Cache(dev, [L], H, D, 16, g)
    c.append(k.to(dev), v.to(dev), [L], [L])
    got = c.attend(q.to(dev), [L], [1]).cpu().double().numpy()
    kq, vq = ref.quantize(k, g), ref.quantize(v, g)
    kv = [(ref.values(*kq, g), ref.values(*vq, g), ref.bf16_f64(kq[1]).max(-1),
           ref.bf16_f64(vq[1]).max(-1))]
    want, parts = ref.attention(q.double().numpy(), kv, [L], [1], D ** -0.5, 0)
    assert (np.abs(got - want) <= ref.bound(want, parts, D)).all()


def test_attention_leaves_out_missing_pages(dev):
    """Page numbers out of range are reported and their keys left out."""
    check_attention(dev, 128, 128, 16, 2, 4, [100, 64], [1, 2], seed=14,
                    holes=[(0, 2, -1), (0, 3, 10 ** 6), (1, 0, -2 ** 31)])
    assert qz.qz_device_status() == 0


def test_append_and_read_of_missing_places(dev):
    """A token without a valid page is dropped, one before position 0 too; the
    rest of the call is done, and the status tells."""
    H, D, g = 2, 64, 32
    k, v = keys((6, H, D), 1), randn((6, H, D), 2)
    c = Cache(dev, [40, 3], H, D, 16, g, fill=0x11)
    c.table[0, 1] = 999
    c.append(k.to(dev), v.to(dev), [18, 1], [4, 2])   # positions 14..17 and -1, 0
    assert qz.qz_device_status() == qz.QZ_ERR_DEVICE_INDEX
    out = c.read([18, 1], [4, 2])
    assert qz.qz_device_status() == qz.QZ_ERR_DEVICE_INDEX
    assert qz.qz_device_status() == 0
    gone = [2, 3, 4]
    for x, got in ((k, out[0]), (v, out[1])):
        w = torch.from_numpy(ref.values(*ref.quantize(x, g), g)).to(torch.bfloat16)
        w[gone] = 0.0
        assert torch.equal(got.cpu(), w)
    host = c.buf.cpu().numpy()
    touched = {c.rows[0][0], c.rows[1][0]}
    page = len(host) // c.pages
    for p in range(c.pages):
        if p not in touched:
            assert (host[p * page:(p + 1) * page] == 0x11).all()
    # a length the page table cannot hold
    c.table[0, 1] = 0
    c.attend(randn((1, H, D), 3).to(dev), [1000, 1], [1, 0])
    assert qz.qz_device_status() == qz.QZ_ERR_DEVICE_INDEX


def test_strided_heads(dev):
    """k, v and q as views of one fused projection, out inside a larger buffer."""
    H, share, D, g, lens, new = 2, 3, 128, 64, [33, 5], [33, 5]
    T = sum(new)
    fused = randn((T, H * share + 2 * H, D), 5).to(dev)
    q, k, v = fused[:, :H * share], fused[:, H * share:H * share + H], fused[:, H * share + H:]
    a, b = Cache(dev, lens, H, D, 16, g), Cache(dev, lens, H, D, 16, g)
    a.append(k, v, lens, new)
    b.append(k.contiguous(), v.contiguous(), lens, new)
    assert torch.equal(a.buf, b.buf)
    wide = torch.zeros((T, H * share + 1, D), dtype=torch.bfloat16, device=dev)
    a.attend(q, lens, new, out=wide[:, 1:])
    want = a.attend(q.contiguous(), lens, new)
    assert torch.equal(wide[:, 1:], want) and (wide[:, 0] == 0).all()


@pytest.mark.parametrize("lens,new", [([40, 3], [2, 1]), ([900], [1])])
def test_results_at_odd_addresses(dev, lens, new):
    """An output array that is only 2-byte aligned, with an odd token stride."""
    H, share, D, g = 1, 3, 64, 64
    c = Cache(dev, lens, H, D, 16, g)
    c.append(keys((sum(lens), H, D), 1).to(dev), randn((sum(lens), H, D), 2).to(dev), lens, lens)
    q = randn((sum(new), share, D), 3).to(dev)
    want = c.attend(q, lens, new)
    wide = torch.zeros(sum(new) * 201 + 7, dtype=torch.bfloat16, device=dev)
    view = wide[7:].view(sum(new), 201)[:, :192].unflatten(1, (share, D))
    c.attend(q, lens, new, out=view)
    assert torch.equal(view, want)
    wide[7:].view(sum(new), 201)[:, :192] = 0
    assert (wide == 0).all()


def test_python_argument_checks(dev):
    lens = [5, 9]
    c = Cache(dev, lens, 2, 64, 16, 64)
    k = randn((14, 2, 64), 1).to(dev)
    ld, cu = i32(lens, dev), i32([0, 5, 14], dev)
    good = dict(cache=c.buf, k=k, v=k, page_table=c.table, kv_lens=ld, cu_tokens=cu, page_size=16,
                group_size=64)
    qz.qz_kv4_append(**good)
    for bad in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=k[:5]), dict(k=k.view(14, 128)),
                dict(k=k.transpose(1, 2)), dict(page_table=c.table.long()), dict(kv_lens=ld[:1]),
                dict(cu_tokens=cu[:2]), dict(cu_tokens=cu.cpu()), dict(page_table=c.table[0]),
                dict(cache=c.buf.view(torch.int8)), dict(k=k.cpu(), v=k.cpu()),
                dict(page_table=c.table[:, ::2])):
        with pytest.raises(ValueError):
            qz.qz_kv4_append(**dict(good, **bad))
    with pytest.raises(ValueError):
        qz.qz_kv4_attention(k, c.buf, c.table, ld, cu, 2, 16, 64, out=k[:5])
    with pytest.raises(ValueError):
        qz.qz_kv4_read(c.buf, c.table, ld, cu, 14, 2, 64, 16, 64, k=k[:5])
    for bad in (dict(page_size=8), dict(group_size=128), dict(cache=c.buf[:64])):
        with pytest.raises(qz.QzError):
            qz.qz_kv4_append(**dict(good, **bad))
    empty = k[:0]
    zero = i32([0, 0, 0], dev)
    qz.qz_kv4_append(c.buf, empty, empty, c.table, ld, zero, 16, 64)
    assert qz.qz_kv4_attention(empty, c.buf, c.table, ld, zero, 2, 16, 64).shape == empty.shape
    assert qz.qz_kv4_read(c.buf, c.table, ld, zero, 0, 2, 64, 16, 64)[0].shape == empty.shape
    assert qz.qz_device_status() == 0


def test_results_repeat_and_counters_return_to_zero(dev):
    lens, new = [4000, 900, 17], [1, 3, 1]
    k, v = keys((sum(lens), 2, 128), 1).to(dev), randn((sum(lens), 2, 128), 2).to(dev)
    c = Cache(dev, lens, 2, 128, 16, 128)
    c.append(k, v, lens, lens)
    q = randn((5, 16, 128), 3).to(dev)
    ws = torch.zeros(qz.qz_workspace_bytes(qz.QZ_OP_KV4_ATTENTION, 1, 1, 128, 0),
                     dtype=torch.uint8, device=dev)
    first = c.attend(q, lens, new, workspace=ws)
    for _ in range(20):
        assert torch.equal(c.attend(q, lens, new, workspace=ws), first)
    assert (ws[:1280] == 0).all()


def test_graph_replay_with_growing_sequences(dev):
    """A captured decode step (append, attend) replayed while the lengths, pages
    and inputs change in place."""
    H, share, D, g, page = 2, 4, 128, 128, 16
    start, steps = [30, 7, 100], 20
    full = [n + steps for n in start]
    c = Cache(dev, full, H, D, page, g)
    k0, v0 = keys((sum(start), H, D), 1), randn((sum(start), H, D), 2)
    c.append(k0.to(dev), v0.to(dev), start, start)
    ws = qz.Workspace(dev)
    lens = i32(start, dev)
    cu = i32([0, 1, 2, 3], dev)
    q, k, v = (torch.zeros((3, n, D), dtype=torch.bfloat16, device=dev) for n in (H * share, H, H))
    out = torch.zeros_like(q)
    ws.get(qz.qz_workspace_bytes(qz.QZ_OP_KV4_ATTENTION, 1, 1, D, 0), ("kv4_attention", D))

    def step():
        lens.add_(1)
        qz.qz_kv4_append(c.buf, k, v, c.table, lens, cu, page, g)
        qz.qz_kv4_attention(q, c.buf, c.table, lens, cu, H, page, g, out=out, workspace=ws)

    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        step()
        lens.sub_(1)
    torch.cuda.current_stream(dev).wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ks, vs = [k0.split(start), v0.split(start)]
    ks, vs = [list(x) for x in (ks, vs)]
    for i in range(steps):
        qi, ki, vi = randn((3, H * share, D), 50 + i), keys((3, H, D), 80 + i), randn((3, H, D), 90 + i)
        q.copy_(qi); k.copy_(ki); v.copy_(vi)
        graph.replay()
        torch.cuda.synchronize()
        kv = []
        for b in range(3):
            ks[b], vs[b] = torch.cat([ks[b], ki[b:b + 1]]), torch.cat([vs[b], vi[b:b + 1]])
            kq, vq = ref.quantize(ks[b], g), ref.quantize(vs[b], g)
            kv.append((ref.values(*kq, g), ref.values(*vq, g), ref.bf16_f64(kq[1]).max(-1),
                       ref.bf16_f64(vq[1]).max(-1)))
        now = [n + i + 1 for n in start]
        want, parts = ref.attention(qi.double().numpy(), kv, now, [1, 1, 1], D ** -0.5, 0)
        got = out.cpu().double().numpy()
        assert (np.abs(got - want) <= ref.bound(want, parts, D)).all(), i
    assert qz.qz_device_status() == 0


def test_side_stream_and_shared_workspace(dev):
    """Calls of different sizes on one stream share a Workspace, beside GEMVs."""
    ws = qz.Workspace(dev)
    st = torch.cuda.Stream(dev)
    cases = []
    for D, g, lens in ((128, 128, [3000]), (64, 32, [40, 2000]), (128, 64, [700] * 5)):
        c = Cache(dev, lens, 2, D, 16, g)
        c.append(keys((sum(lens), 2, D), D).to(dev), randn((sum(lens), 2, D), 3).to(dev), lens, lens)
        q = randn((len(lens), 8, D), 4).to(dev)
        cases.append((c, q, lens, c.attend(q, lens, [1] * len(lens))))
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        lens_dev = [(i32(l, dev), i32(list(range(len(l) + 1)), dev)) for _, _, l, _ in cases]
    for _ in range(3):
        for (c, q, lens, want), (ld, cu) in zip(cases, lens_dev):
            got = qz.qz_kv4_attention(q, c.buf, c.table, ld, cu, 2, 16, c.g, workspace=ws, stream=st)
            st.synchronize()
            assert torch.equal(got, want)


def test_cache_past_4_gb(dev):
    """Pages whose byte offsets do not fit in 32 bits."""
    H, D, g, page = 8, 256, 64, 256
    per = qz.qz_kv4_cache_bytes(1, H, D, page, g)
    pages = (9 << 29) // per + 3                     # 4.5 GB
    buf = torch.empty(pages * per, dtype=torch.uint8, device=dev)
    lens = [300, 200]
    rows = [[pages - 1, pages - 3], [pages - 2, 0]]
    c = Cache(dev, lens, H, D, page, g)
    k, v = keys((500, H, D), 1).to(dev), randn((500, H, D), 2).to(dev)
    c.append(k, v, lens, lens)
    q = randn((2, 16, D), 3).to(dev)
    want = c.attend(q, lens, [1, 1])
    c.buf, c.table = buf, i32(rows, dev)
    c.append(k, v, lens, lens)
    assert torch.equal(c.attend(q, lens, [1, 1]), want)
    assert qz.qz_device_status() == 0


def test_infinite_and_nan_queries(dev):
    """A row with an infinity or a NaN gives NaN; its neighbours are untouched."""
    lens, H, D = [50], 1, 128
    c = Cache(dev, lens, H, D, 16, 128)
    c.append(keys((50, H, D), 1).to(dev), randn((50, H, D), 2).to(dev), lens, lens)
    q = randn((1, 8, D), 3)
    clean = c.attend(q.to(dev), lens, [1])
    q[0, 2, 5] = float("nan")
    q[0, 4, 7] = float("inf")
    got = c.attend(q.to(dev), lens, [1])
    assert got[0, 2].isnan().all() and got[0, 4].isnan().all()
    keep = [0, 1, 3, 5, 6, 7]
    assert torch.equal(got[0, keep], clean[0, keep])


def attend_values(dev, k, v, q, new, g, window=0):
    """Attention over one sequence, and the 64-bit form over its finite tokens
    (what stands at the others must not be seen by the rows compared)."""
    L, H, D = k.shape
    c = Cache(dev, [L], H, D, 16, g)
    c.append(k.to(dev), v.to(dev), [L], [L])
    got = c.attend(q.to(dev), [L], [new], window=window).cpu().double().numpy()
    fine = [torch.where(x.isfinite().all(-1, keepdim=True), x, torch.zeros_like(x)) for x in (k, v)]
    kq, vq = ref.quantize(fine[0], g), ref.quantize(fine[1], g)
    kv = [(ref.values(*kq, g), ref.values(*vq, g), ref.bf16_f64(kq[1]).max(-1),
           ref.bf16_f64(vq[1]).max(-1))]
    want, parts = ref.attention(q.double().numpy(), kv, [L], [new], D ** -0.5, window)
    return got, want, ref.bound(want, parts, D)


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e25])
@pytest.mark.parametrize("which", ["k", "v"])
def test_keys_a_row_may_not_see_change_nothing(dev, D, g, value, which):
    """The last token holds a value that only the last query may see, the first
    one a value that the window hides from all."""
    L, new = 40, 3
    k, v = keys((L, 1, D), 21), randn((L, 1, D), 22)
    x = k if which == "k" else v
    x[L - 1, 0, 5] = value
    x[0, 0, 7] = value
    got, want, lim = attend_values(dev, k, v, randn((new, 2, D), 23), new, g, window=30)
    assert (np.abs(got - want)[:new - 1] <= lim[:new - 1]).all()
    if value == float("inf"):              # a NaN is left out by quantize_pack: its scale is finite
        assert not np.isfinite(got[new - 1]).all()


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("power", [-40, -20, 20, 40])
def test_rows_of_values_of_different_sizes(dev, D, g, power):
    """Heads of one tile that look at keys whose values differ in size by far."""
    L = 40
    k, v = torch.zeros(L, 1, D), randn((L, 1, D), 31).float()
    k[3, 0, :D // 2], k[35, 0, D // 2:] = 4.0, 4.0
    v[35] *= 2.0 ** power
    q = torch.zeros(1, 2, D)
    q[0, 0, :D // 2], q[0, 1, D // 2:] = 3.0, 3.0
    k, v, q = (t.to(torch.bfloat16) for t in (k, v, q))
    got, want, lim = attend_values(dev, k, v, q, 1, g)
    assert (np.abs(got - want) <= lim).all()


@pytest.mark.parametrize("D,g", ref.COMBOS)
@pytest.mark.parametrize("late", [20, 50, 90])
def test_a_later_key_of_small_values_takes_the_weight(dev, D, g, late):
    """Large values at the first keys, then a key with nearly all the weight and
    small values, in the same step or in a later one of the same warp."""
    L = 100
    k, v = torch.zeros(L, 1, D), randn((L, 1, D), 41).float()
    k[late] = 4.0
    v[:8] *= 2.0 ** 20
    v[late] *= 2.0 ** -4
    q = torch.full((1, 1, D), 96.0 / D ** 0.5 / 4)
    k, v, q = (t.to(torch.bfloat16) for t in (k, v, q))
    got, want, lim = attend_values(dev, k, v, q, 1, g)
    assert (np.abs(got - want) <= lim).all()


def test_scores_far_below_zero(dev):
    """Every score of a row near -1e35: the softmax is that of their differences
    (one key in front by far), not that of a row without keys."""
    H, D, g, L = 1, 128, 128, 20
    k, v = torch.full((L, H, D), 1e17), randn((L, H, D), 51)
    k[7] = 5e16
    k = k.to(torch.bfloat16)
    c = Cache(dev, [L], H, D, 16, g)
    c.append(k.to(dev), v.to(dev), [L], [L])
    q = torch.full((1, 2, D), -1e17, dtype=torch.bfloat16)
    got = c.attend(q.to(dev), [L], [1]).cpu().double().numpy()
    vq = ref.quantize(v, g)
    want = ref.values(*vq, g)[7]
    S = ref.bf16_f64(vq[1]).max()
    # P is 1 at key 7 and 0 elsewhere: one weight S of 2^-11, and bf16's half step
    assert (np.abs(got[0] - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * np.abs(want) + 2.0 ** -20 * S).all()
