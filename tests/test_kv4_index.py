"""CPU checks of the paged cache's index arithmetic and the attention's work
split (csrc/qz_kv4_index.cuh, compiled here with the host compiler), and of the
host-side refusals of the qz_kv4 entry points."""
import ctypes
import os
import random
import subprocess

import numpy as np
import pytest

import kv4_ref as ref
import weight_only_quantization_wise_b200 as qz

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SHIM = r"""
#include "qz_kv4_index.cuh"
using namespace qz::kv4;
typedef long long ll;
extern "C" {
int s_record_bytes(int D, int g) { return (int)record_bytes(D, g); }
int s_word_byte(int w, int gid, int tid) { return word_byte(w, gid, tid); }
int s_k_word_byte(int D, int t, int c8) { return k_word_byte(D, t, c8); }
int s_v_unit_byte(int D, int t, int w, int hi, int gid) { return v_unit_byte(D, t, w, hi, gid); }
int s_off(int D, int ng, int which) {
    const int o[6] = {k_codes_off(), v_codes_off(D), k_scales_off(D), v_scales_off(D, ng),
                      k_zeros_off(D, ng), v_zeros_off(D, ng)};
    return o[which];
}
ll s_record_index(const int *row, ll max_pages, ll num_pages, int heads, int h, int pb, int block) {
    return record_index(row, max_pages, num_pages, heads, h, pb, block);
}
void s_store_work(int cu0, int cu1, int len, int T, int heads, ll *o) {
    const StoreWork s = store_work(cu0, cu1, len, T, heads);
    o[0] = s.n; o[1] = s.block0; o[2] = s.blocks; o[3] = s.first; o[4] = s.units;
}
void s_block_range(int cu0, int cu1, int len, int T, int block, int *o) {
    const StoreWork s = store_work(cu0, cu1, len, T, 1);
    o[0] = block_lo(s, block); o[1] = block_hi(s, block);
}
void s_seq_work(int cu0, int cu1, int len, int T, int cap, int win, int share, int heads, int rows,
                ll *o) {
    const SeqWork s = seq_work(cu0, cu1, len, T, cap, win, share, heads, rows);
    o[0] = s.n; o[1] = s.len; o[2] = s.block0; o[3] = s.blocks; o[4] = s.row_tiles; o[5] = s.units;
}
ll s_range_begin(ll c, ll q, ll u) { return range_begin(c, q, u); }
ll s_cta_quota(ll u, ll items, int blocks, ll c, int m, int w) {
    return cta_quota(u, items, blocks, c, m, w);
}
ll s_quotient(ll a, ll b) { return quotient(a, b); }
int s_warp_quota(ll n, int w) { return warp_quota(n, w); }
int s_partial_slot(ll a, ll b) { return partial_slot(a, b); }
}
"""


@pytest.fixture(scope="module")
def ix(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv4")
    src, lib = d / "shim.cpp", d / "shim.so"
    src.write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "weight_only_quantization_wise_b200", "csrc"), str(src),
                    "-o", str(lib)], check=True)
    so = ctypes.CDLL(str(lib))
    ll = ctypes.c_longlong
    for name, args in (("s_record_index", [ctypes.c_void_p, ll, ll] + [ctypes.c_int] * 4),
                       ("s_range_begin", [ll, ll, ll]), ("s_quotient", [ll, ll]),
                       ("s_cta_quota", [ll, ll, ctypes.c_int, ll, ctypes.c_int, ctypes.c_int])):
        f = getattr(so, name)
        f.argtypes, f.restype = args, ll
    so.s_seq_work.argtypes = [ctypes.c_int] * 9 + [ctypes.c_void_p]
    so.s_warp_quota.argtypes = [ll, ctypes.c_int]
    so.s_partial_slot.argtypes = [ll, ll]
    so.s_store_work.argtypes = [ctypes.c_int] * 5 + [ctypes.c_void_p]
    so.s_block_range.argtypes = [ctypes.c_int] * 5 + [ctypes.c_void_p]
    return so


@pytest.mark.parametrize("D,g", ref.COMBOS)
def test_record_layout(ix, D, g):
    """The index header's places are the documented ones, every code has a
    nibble of its own, and the parts fill the record without gaps."""
    ng = D // g
    assert ix.s_record_bytes(D, g) == ref.record_size(D, g) and ref.record_size(D, g) % 16 == 0
    assert [ix.s_off(D, ng, i) for i in range(6)] == [
        0, 8 * D, 16 * D, 16 * D + 32 * ng, 16 * D + 64 * ng, 16 * D + 80 * ng]
    seen = set()
    for t in range(16):
        for d in range(D):
            byte, high = ref.k_place(D, t, d)
            assert byte == ix.s_k_word_byte(D, t, d // 8) + d % 8 // 2 and high == d % 2
            seen.add((byte, high))
            byte, high = ref.v_place(D, t, d)
            n = d % 64 // 16
            assert byte == 8 * D + ix.s_v_unit_byte(D, t, d // 64, d % 16 // 8, d % 8) + n // 2
            assert high == n % 2
            seen.add((byte, high))
    assert seen == {(b, h) for b in range(16 * D) for h in (0, 1)}


@pytest.mark.parametrize("D", [64, 128, 256])
def test_lane_words(ix, D):
    """What a lane finds in the 16-byte pieces it loads is its MMA operand:
    tokens gid and gid + 8 for the keys, tokens 8 p + 2 tid, + 1 and rows
    gid, gid + 8 of each 16-row tile for the values."""
    kw = D // 32
    for lane in range(32):
        gid, tid = lane // 4, lane % 4
        for q in range(2 * kw // 4):
            for x in range(4):
                word, byte = 4 * q + x, q * 512 + lane * 16 + 4 * x
                assert byte == ix.s_word_byte(word, gid, tid)
                hi, j = word // kw, word % kw
                assert byte == ix.s_k_word_byte(D, 8 * hi + gid, 4 * j + tid)
                p, hi, w = word // kw, word % kw // (D // 64), word % (D // 64)
                for half in (0, 1):
                    assert byte + 2 * half == ix.s_v_unit_byte(D, 8 * p + 2 * tid + half, w, hi,
                                                               gid)


def test_bad_pages_have_no_record(ix):
    rng = random.Random(5)
    for _ in range(200):
        max_pages, num_pages, heads = rng.randint(1, 9), rng.randint(1, 30), rng.randint(1, 5)
        pb = rng.choice([1, 2, 3, 4, 8])
        table = np.array([rng.choice([-1, -2 ** 31, num_pages, 2 ** 31 - 1,
                                      rng.randrange(num_pages), rng.randrange(num_pages)])
                          for _ in range(max_pages)], np.int32)
        for block in range(-2, max_pages * pb + 3):
            h = rng.randrange(heads)
            got = ix.s_record_index(table.ctypes.data, max_pages, num_pages, heads, h, pb, block)
            inside = 0 <= block < max_pages * pb
            if not inside or not 0 <= table[block // pb] < num_pages:
                assert got == -1
            else:
                assert got == (int(table[block // pb]) * heads + h) * pb + block % pb
                assert 0 <= got < num_pages * heads * pb


def test_record_offsets_past_32_bits(ix):
    table = np.array([2 ** 31 - 2], np.int32)
    got = ix.s_record_index(table.ctypes.data, 1, 2 ** 31 - 1, 8, 7, 4, 3)
    assert got == ((2 ** 31 - 2) * 8 + 7) * 4 + 3


def test_quotient(ix):
    for a, b in [(0, 1), (7, 7), (2 ** 32 - 1, 3), (2 ** 32, 3), (2 ** 40 + 5, 2 ** 33), (9, 2 ** 35)]:
        assert ix.s_quotient(a, b) == a // b


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 40])
@pytest.mark.parametrize("length", [0, 1, 5, 15, 16, 17, 31, 32, 100, 2 ** 31 - 1, -3])
def test_store_work_covers_each_token_once(ix, n, length):
    """The tokens' positions, cut into blocks of 16: each position is in one
    block's range, also positions in front of 0."""
    o, r = (ctypes.c_longlong * 5)(), (ctypes.c_int * 2)()
    ix.s_store_work(7, 7 + n, length, 1000, 3, o)
    assert o[0] == n and o[3] == length - n and o[4] == 3 * o[2]
    seen = []
    for block in range(o[1], o[1] + o[2]):
        ix.s_block_range(7, 7 + n, length, 1000, block, r)
        assert 0 <= r[0] < r[1] <= 16
        seen += [block * 16 + t for t in range(r[0], r[1])]
    assert seen == list(range(length - n, length))
    assert o[2] <= n // 16 + 2


def batches():
    rng = random.Random(7)
    for _ in range(60):
        B = rng.choice([1, 1, 2, 5, 40, 300])
        new = [rng.choice([0, 1, 1, 1, 3, rng.randint(0, 70)]) for _ in range(B)]
        lens = [rng.choice([0, 1, 15, 16, 17, rng.randint(0, 3000), n]) for n in new]
        yield (lens, new, rng.choice([0, 0, 1, 16, 17, 900]), rng.choice([1, 2, 3, 4, 8, 16]),
               rng.choice([1, 2, 8]), rng.choice([8, 16]), rng.choice([1, 3, 296]),
               rng.choice([1, 32]), rng.choice([3, 4, 6, 8]))


@pytest.mark.parametrize("case", list(range(60)))
def test_work_split(ix, case):
    """Every unit belongs to one warp of one CTA; each item that several CTAs
    share has one part in each of them, in distinct slots of the workspace, and
    is counted at a CTA that counts no other item; every key that a row sees
    lies in a unit."""
    lens, new, window, share, heads, rows, grid, min_units, warps = list(batches())[case]
    items, cu, T = [], 0, max(1, sum(new))
    for L, n in zip(lens, new):
        o = (ctypes.c_longlong * 6)()
        ix.s_seq_work(cu, cu + n, L, T, 4096, window, share, heads, rows, o)
        cu += n
        assert o[0] == n and o[1] == L and o[5] == o[4] * heads * o[3]
        assert o[4] == -(-n * share // rows)
        items += [int(o[3])] * int(o[4] * heads)
        for i in range(n):                                   # keys of each row
            p = L - n + i
            first = max(0, p - window + 1) if window else 0
            if p >= 0:
                assert o[2] * 16 <= first and p < (o[2] + o[3]) * 16
    units = sum(items)
    if units == 0:
        return
    begins = np.cumsum([0] + items)
    quota = ix.s_cta_quota(units, len(items), max(items), grid, min_units, 96)
    assert quota * grid >= units
    if len(set(items)) == 1 and items[0] <= 96 and len(items) <= grid:
        assert quota == items[0]                         # whole items
    else:
        assert quota >= min_units
    covered, homes, slots, active = 0, {}, {}, 0
    for c in range(grid):
        b0, b1 = ix.s_range_begin(c, quota, units), ix.s_range_begin(c + 1, quota, units)
        if b0 >= b1:
            assert b0 == units
            continue
        assert b0 == covered and c == active
        active += 1
        assert all(u // quota == c for u in (b0, (b0 + b1) // 2, b1 - 1))
        wq = ix.s_warp_quota(b1 - b0, warps)
        assert wq % 2 == 0 and wq * warps >= b1 - b0
        covered = b1
        first = int(np.searchsorted(begins, b0, "right") - 1)
        last = int(np.searchsorted(begins, b1 - 1, "right") - 1)
        for it in {first, last}:
            i0, i1 = int(begins[it]), int(begins[it + 1])
            if i0 >= b0 and i1 <= b1:
                continue
            home = i0 // quota
            assert homes.setdefault(home, it) == it
            slot = ix.s_partial_slot(i0, b0)
            assert (c, slot) not in slots
            slots[(c, slot)] = it
            # how the last to arrive finds this part
            s0 = ix.s_partial_slot(i0, ix.s_range_begin(home, quota, units))
            assert slot == (s0 if c == home else 0)
    assert covered == units
    for home, it in homes.items():
        c1 = (int(begins[it + 1]) - 1) // quota
        assert sorted(c for (c, _), i in slots.items() if i == it) == list(range(home, c1 + 1))


def test_wild_lengths_and_offsets_stay_in_range(ix):
    """Values no caller should pass: work counts stay non-negative and bounded."""
    big = 2 ** 31 - 1
    for cu0, cu1, L in [(0, big, 5), (-big, 5, 5), (5, 0, 5), (-1, 3, 5), (0, 1, -big), (0, 1, big),
                        (big - 1, big, big)]:
        for window in (0, 1, 1000):
            o = (ctypes.c_longlong * 6)()
            ix.s_seq_work(cu0, cu1, L, 100, 2 ** 31 - 32, window, 16, 8, 8, o)
            n, length, block0, blocks, tiles, units = o
            assert 0 <= n <= 100 and 0 <= length <= 2 ** 31 - 32 and blocks >= 1
            assert 0 <= block0 and (block0 + blocks) * 16 < 2 ** 31
            assert tiles == -(-n * 16 // 8) and units == tiles * 8 * blocks


# ---------------------------------------------------------------------------
# refusals (fake addresses that are never dereferenced)
# ---------------------------------------------------------------------------
OK, INVALID, ALIGN, UNSUP, WS = 0, 1, 2, 3, 4
A, Bp, C, D4, E, F, W = (ctypes.c_void_p(0x10000 * i) for i in range(1, 8))
MIS = ctypes.c_void_p(0x10002)
GOOD = dict(T=3, B=2, heads=8, D=128, page=16, g=128, pages=4, width=2)


def shape(**kw):
    v = dict(GOOD, **kw)
    return tuple(v[k] for k in ("T", "B", "heads", "D", "page", "g", "pages", "width"))


BAD_SHAPES = [(dict(T=0), INVALID), (dict(B=0), INVALID), (dict(heads=0), INVALID),
              (dict(D=96), UNSUP), (dict(D=0), INVALID), (dict(g=48), UNSUP),
              (dict(g=0), INVALID), (dict(D=64, g=128), UNSUP), (dict(D=256, g=32), UNSUP),
              (dict(page=8), UNSUP), (dict(page=0), INVALID), (dict(page=24), UNSUP),
              (dict(page=65552), UNSUP), (dict(pages=0), INVALID), (dict(width=0), INVALID),
              (dict(T=2 ** 31), INVALID), (dict(T=2 ** 30), INVALID), (dict(B=2 ** 21), INVALID)]


def append(cache=A, k=Bp, v=C, ks=1024, vs=1024, pt=D4, kl=E, cu=F, **kw):
    return qz.lib.qz_kv4_append(cache, k, v, ks, vs, pt, kl, cu, *shape(**kw), None)


def read(cache=A, k=Bp, v=C, pt=D4, kl=E, cu=F, **kw):
    return qz.lib.qz_kv4_read(cache, pt, kl, cu, *shape(**kw), k, v, None)


def attend(q=Bp, qs=4096, cache=A, pt=D4, kl=E, cu=F, q_heads=32, scale=0.1, window=0, out=C,
           os=4096, ws=W, wb=1 << 30, **kw):
    T, B, H, D, page, g, pages, width = shape(**kw)
    return qz.lib.qz_kv4_attention(q, qs, cache, pt, kl, cu, T, B, q_heads, H, D, page, g, pages,
                                   width, scale, window, out, os, ws, wb, None)


@pytest.mark.parametrize("kw,expect", BAD_SHAPES)
def test_kv4_shapes_are_refused(kw, expect):
    wide = dict(ks=1 << 30, vs=1 << 30)
    assert append(**wide, **kw) == expect
    assert read(**kw) == expect
    assert attend(qs=1 << 30, os=1 << 30, **kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(cache=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(pt=None), INVALID), (dict(kl=None), INVALID), (dict(cu=None), INVALID),
    (dict(cache=MIS), ALIGN), (dict(k=MIS), ALIGN), (dict(v=MIS), ALIGN), (dict(pt=MIS), ALIGN),
    (dict(ks=1023), INVALID), (dict(vs=0), INVALID), (dict(ks=1028), ALIGN),
])
def test_kv4_append_refuses(kw, expect):
    assert append(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(cache=None), INVALID), (dict(k=None), INVALID), (dict(v=MIS), ALIGN),
    (dict(kl=MIS), ALIGN), (dict(cu=MIS), ALIGN),
])
def test_kv4_read_refuses(kw, expect):
    assert read(**kw) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(q=MIS), ALIGN),
    (dict(out=ctypes.c_void_p(0x10001)), ALIGN), (dict(q_heads=20), INVALID),
    (dict(q_heads=0), INVALID), (dict(window=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(qs=4095), INVALID), (dict(qs=4100), ALIGN),
    (dict(os=100), INVALID), (dict(ws=None), WS), (dict(wb=1000), WS),
    (dict(ws=ctypes.c_void_p(0x70010)), ALIGN),
])
def test_kv4_attention_refuses(kw, expect):
    assert attend(**kw) == expect


def test_kv4_sizes():
    for D, g in ref.COMBOS:
        assert qz.qz_kv4_cache_bytes(7, 3, D, 48, g) == 7 * 3 * 3 * ref.record_size(D, g)
    with pytest.raises(qz.QzError):
        qz.qz_kv4_cache_bytes(7, 3, 128, 40, 128)
    with pytest.raises(qz.QzError):
        qz.qz_kv4_cache_bytes(2 ** 31 - 1, 65536, 256, 65536, 64)
    # two slots of 16 rows (head_dim + 4 fp32, 2 fp32 per row) and a counter
    # for each of 2 x 148 CTAs
    for D in (64, 128, 256):
        assert (qz.qz_workspace_bytes(qz.QZ_OP_KV4_ATTENTION, 1, 1, D, 0) ==
                1280 + 296 * 2 * 16 * (D + 6) * 4)
    with pytest.raises(qz.QzError):
        qz.qz_workspace_bytes(qz.QZ_OP_KV4_ATTENTION, 1, 1, 96, 0)
    assert qz.qz_status_string(qz.QZ_ERR_DEVICE_INDEX) != "unknown status"
