// qz_kv4.cu -- the paged 4-bit key/value cache: append (quantize), read
// (dequantize) and attention over it.
//
// The cache holds the int4 asymmetric group format of qz_quantize_pack per
// (token, head): codes c, a bf16 scale S and a zero-point Z per group of g of
// the head's D values, standing for S (c - Z).  Layout and work split:
// qz_kv4_index.cuh.
#include <cuda_runtime.h>

#include "qz_kv4_index.cuh"
#include "qz_sm100.cuh"

namespace qz {
namespace {

using namespace sm100;
using namespace kv4;

constexpr unsigned kErrIndex = 2u;     // bit of the device error word: bad page or position

// ---------------------------------------------------------------------------
// append: one warp per (token, key head)
// ---------------------------------------------------------------------------
struct StoreArgs {
    const uint16_t *k, *v;             // append: input; read: unused
    uint16_t *k_out, *v_out;           // read
    int64_t k_stride, v_stride;        // elements between tokens
    uint8_t *cache;
    const int32_t *page_table, *kv_lens, *cu;
    int64_t T, B, max_pages, num_pages;
    int kv_heads, page_size;
    unsigned int *err_word;
};

constexpr int kStoreWarps = 8;

// Token t's place: its sequence's page-table row and position, false for a
// token behind the last sequence.
__device__ __forceinline__ bool locate(const StoreArgs &p, int64_t t, int64_t &b, int64_t &pos) {
    b = find_sequence(p.cu, p.B, t);
    if (b < 0) return false;
    pos = (int64_t)p.kv_lens[b] - ((int64_t)p.cu[b + 1] - t);
    return true;
}

// Scale, zero and codes as qz_quantize_pack forms them (qz.h: range widened
// to 0, S = (max - min) / 15 in fp32 stored as bf16 rounded up, 0 -> 1).
// code = clamp(round(x / S + Z)): with r = 1/S rounded, fma(x, r, Z + 192)
// lies on the same side of every half-way point as x / S + Z (bf16 x and S
// keep x / S + Z at least 2^-10 from a half-way point it does not hit; the
// argument is written out at chunk_codes in qz_quantize.cu), and adding
// 1.5 2^23 - 192 rounds half to even into the low mantissa bits.
__device__ __forceinline__ uint32_t code4(float x, float s, float r, float z) {
    if (!(r < __int_as_float(0x7F800000))) {        // 1/S overflows: IEEE division
        const int q = (int)rintf(__fadd_rn(__fdiv_rn(x, s), z));
        return (uint32_t)min(max(q, 0), 15);
    }
    const float y = __fmaf_rn(x, r, __fadd_rn(z, 192.0f));
    const uint32_t b = __float_as_uint(__fadd_rn(y, 12582912.0f - 192.0f));
    return min(b, 0x4B40000Fu) & 15u;
}

template <int D, int G>
__device__ __forceinline__ void quantize_head(const uint16_t *src, int lane, uint8_t *codes,
                                              uint16_t *scales, uint8_t *zeros) {
    constexpr int V = D / 32;                        // values per lane, consecutive
    constexpr int LPG = G / V;                       // lanes per group
    float x[V];
    if constexpr (V == 2) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(src)[lane];
        x[0] = dev::bf16_lo(w); x[1] = dev::bf16_hi(w);
    } else if constexpr (V == 4) {
        const uint2 w = reinterpret_cast<const uint2 *>(src)[lane];
        x[0] = dev::bf16_lo(w.x); x[1] = dev::bf16_hi(w.x);
        x[2] = dev::bf16_lo(w.y); x[3] = dev::bf16_hi(w.y);
    } else {
        const uint4 w = reinterpret_cast<const uint4 *>(src)[lane];
        x[0] = dev::bf16_lo(w.x); x[1] = dev::bf16_hi(w.x);
        x[2] = dev::bf16_lo(w.y); x[3] = dev::bf16_hi(w.y);
        x[4] = dev::bf16_lo(w.z); x[5] = dev::bf16_hi(w.z);
        x[6] = dev::bf16_lo(w.w); x[7] = dev::bf16_hi(w.w);
    }
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) { lo = fminf(lo, x[i]); hi = fmaxf(hi, x[i]); }
#pragma unroll
    for (int o = 1; o < LPG; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    }
    float s = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
    if (s == 0.0f) s = 1.0f;
    const uint32_t sb = dev::bf16_round_up_bits(s);
    s = __uint_as_float(sb << 16);
    const float z = -rintf(__fdiv_rn(lo, s));
    const float r = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < V; ++i) codes[lane * V + i] = (uint8_t)code4(x[i], s, r, z);
    if ((lane & (LPG - 1)) == 0) {
        scales[16 * (lane / LPG)] = (uint16_t)sb;
        zeros[16 * (lane / LPG)] = (uint8_t)(int)z;
    }
}

template <int D, int G>
__global__ void __launch_bounds__(32 * kStoreWarps) kv4_append_kernel(const StoreArgs p) {
    constexpr int NG = D / G;
    __shared__ __align__(16) uint8_t buf[kStoreWarps][D];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kStoreWarps + w;
    if (item >= p.T * p.kv_heads) return;
    const int64_t t = item / p.kv_heads;
    const int h = (int)(item - t * p.kv_heads);
    int64_t b, pos;
    if (!locate(p, t, b, pos)) return;
    int64_t rec = -1;
    if (pos >= 0)
        rec = record_index(p.page_table + b * p.max_pages, p.max_pages, p.num_pages, p.kv_heads,
                           h, p.page_size / kBlock, pos / kBlock);
    if (rec < 0) {
        if (lane == 0) atomicOr(p.err_word, kErrIndex);
        return;
    }
    uint8_t *r = p.cache + rec * record_bytes(D, G);
    const int tk = (int)(pos % kBlock);
    uint8_t *c = buf[w];
    quantize_head<D, G>(p.k + t * p.k_stride + (int64_t)h * D, lane, c,
                        reinterpret_cast<uint16_t *>(r + k_scales_off(D)) + tk,
                        r + k_zeros_off(D, NG) + tk);
    __syncwarp();
    if (lane < D / 8) {
        const uint2 v = reinterpret_cast<const uint2 *>(c)[lane];
        uint32_t lo = v.x | (v.x >> 4), hi = v.y | (v.y >> 4);   // nibble pairs in bytes 0 and 2
        lo = (lo & 0xFFu) | ((lo >> 8) & 0xFF00u);
        hi = (hi & 0xFFu) | ((hi >> 8) & 0xFF00u);
        *reinterpret_cast<uint32_t *>(r + k_codes_off() + k_word_byte(D, tk, lane)) =
            lo | (hi << 16);
    }
    __syncwarp();
    quantize_head<D, G>(p.v + t * p.v_stride + (int64_t)h * D, lane, c,
                        reinterpret_cast<uint16_t *>(r + v_scales_off(D, NG)) + tk,
                        r + v_zeros_off(D, NG) + tk);
    __syncwarp();
    for (int u = lane; u < D / 4; u += 32) {
        const int gid = u & 7, hi = (u >> 3) & 1, wi = u >> 4;
        uint32_t v = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) v |= (uint32_t)c[64 * wi + 16 * n + 8 * hi + gid] << (4 * n);
        *reinterpret_cast<uint16_t *>(r + v_codes_off(D) + v_unit_byte(D, tk, wi, hi, gid)) =
            (uint16_t)v;
    }
}

// ---------------------------------------------------------------------------
// read: one warp per (token, key head); lane l < D / 8 gives d = 8 l .. 8 l + 7
// ---------------------------------------------------------------------------
template <int D, int G>
__global__ void __launch_bounds__(32 * kStoreWarps) kv4_read_kernel(const StoreArgs p) {
    constexpr int NG = D / G;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kStoreWarps + w;
    if (item >= p.T * p.kv_heads) return;
    const int64_t t = item / p.kv_heads;
    const int h = (int)(item - t * p.kv_heads);
    int64_t b, pos;
    if (!locate(p, t, b, pos)) return;
    if (lane >= D / 8) return;
    uint16_t *ko = p.k_out + item * D + 8 * lane, *vo = p.v_out + item * D + 8 * lane;
    int64_t rec = -1;
    if (pos >= 0)
        rec = record_index(p.page_table + b * p.max_pages, p.max_pages, p.num_pages, p.kv_heads,
                           h, p.page_size / kBlock, pos / kBlock);
    if (rec < 0) {
        *reinterpret_cast<uint4 *>(ko) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4 *>(vo) = make_uint4(0u, 0u, 0u, 0u);
        if (lane == 0) atomicOr(p.err_word, kErrIndex);
        return;
    }
    const uint8_t *r = p.cache + rec * record_bytes(D, G);
    const int tk = (int)(pos % kBlock);
    const int grp = 8 * lane / G;
    uint32_t kc = *reinterpret_cast<const uint32_t *>(r + k_word_byte(D, tk, lane));
    uint32_t vc = 0;
    const int wi = lane >> 3, n = (lane >> 1) & 3, hi = lane & 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t u = *reinterpret_cast<const uint16_t *>(r + v_codes_off(D) +
                                                               v_unit_byte(D, tk, wi, hi, i));
        vc |= ((u >> (4 * n)) & 15u) << (4 * i);
    }
    const int so = 16 * grp + tk;
    const float ks = __uint_as_float(
        (uint32_t)reinterpret_cast<const uint16_t *>(r + k_scales_off(D))[so] << 16);
    const float vs = __uint_as_float(
        (uint32_t)reinterpret_cast<const uint16_t *>(r + v_scales_off(D, NG))[so] << 16);
    const int kz = r[k_zeros_off(D, NG) + so], vz = r[v_zeros_off(D, NG) + so];
    uint32_t ko2[4], vo2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int a = (int)((kc >> (8 * i)) & 15u) - kz, c = (int)((kc >> (8 * i + 4)) & 15u) - kz;
        const int e = (int)((vc >> (8 * i)) & 15u) - vz, f = (int)((vc >> (8 * i + 4)) & 15u) - vz;
        ko2[i] = dev::pack_bf16x2(ks * (float)a, ks * (float)c);
        vo2[i] = dev::pack_bf16x2(vs * (float)e, vs * (float)f);
    }
    *reinterpret_cast<uint4 *>(ko) = make_uint4(ko2[0], ko2[1], ko2[2], ko2[3]);
    *reinterpret_cast<uint4 *>(vo) = make_uint4(vo2[0], vo2[1], vo2[2], vo2[3]);
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// Row i of a sequence with n queries and len keys stands at position
// p = len - n + i and sees keys j <= p (and j > p - window):
//   s_j = scale sum_d q_d S_j (c_jd - Z_j),  P = softmax(s),
//   out_d = sum_j P_j S_j (c_jd - Z_j).
// The codes enter the tensor cores as the exact fp16 integers c - Z.  Of a
// 16-bit half, nibble 0 ORed under fp16 1024 is 1024 + c and nibble 1 under 64
// is 64 + c (one LOP3 each for the same nibble of both halves), and one packed
// subtraction of 1024 + Z or 64 + Z leaves c - Z; a shift by 8 does the other
// two.  (Leaving the subtraction out -- codes as fp16 subnormals, Z taken off
// the sums -- saves 4 instructions per word, but the tensor core aligns a
// subnormal's products by its nominal exponent and loses their low bits:
// 2^-15 of the largest product, seen where one key holds the weight and c = Z.)
// Queries are bf16 brought into fp16's range by a power of two per row (exact
// above 2^-24 of the row's largest value).  S stays out of the first product.
// Weights P_j S_j are rounded once to fp16 (relative 2^-12) for the second
// product, scaled by 2^-n, n a running maximum of s_j + log2 of S_j's binade
// beside the softmax's running maximum m of s_j (both in powers of two), so
// that they lie in (0, 2^5) whatever the sizes of V.
// Sums, maxima and partial results are fp32.
struct AttnArgs {
    const uint16_t *q;
    int64_t q_stride;                  // elements between tokens
    const uint8_t *cache;
    const int32_t *page_table, *kv_lens, *cu;
    int64_t T, B, max_pages, num_pages, window, capacity;
    int kv_heads, share, page_blocks;
    float scale_log2;                  // scale * log2(e)
    uint16_t *out;
    int64_t out_stride;
    float *partials;                   // [ctas][2][Slot]
    uint32_t *counters;                // [ctas]
    int64_t min_units;
    uint64_t wait_limit;
    unsigned int *err_word;
};

constexpr float kNoMax = -1e30f;       // running maximum before any key

// A partial result of a row tile: [R][D + 4] fp32 sums, then m, n, l per row.
template <int D, int NB>
struct Slot {
    static constexpr int R = 8 * NB;
    static constexpr int pitch = D + 4;                    // floats: rows 8 apart in banks
    static constexpr int stats = R * pitch;                // [3][R]
    static constexpr int floats = R * pitch + 4 * R;
    static constexpr int bytes = floats * 4;
};

// Dynamic shared memory of a CTA so that two fit on an SM (228 KB, 1 KB of it
// reserved per CTA, and up to 3 KB of static arrays).
constexpr int kAttnSmem = 110 * 1024;

template <int D, int G, int NB, int WARPS>
struct AttnLayout {
    static constexpr int NG = D / G;
    static constexpr int rec = (int)record_bytes(D, G);
    static constexpr int slot = Slot<D, NB>::bytes;
    static constexpr int ring_bytes(int s) { return ((s * rec > slot ? s * rec : slot) + 15) & ~15; }
    static constexpr int total(int s) { return WARPS * (ring_bytes(s) + slot + 8 * s); }
    // records in flight per warp: up to 6, as many as let two CTAs share an SM
    static constexpr int S = total(6) <= kAttnSmem ? 6 : total(5) <= kAttnSmem ? 5
                             : total(4) <= kAttnSmem ? 4 : 3;
    static constexpr int ring = ring_bytes(S);
    static constexpr int ring_off = 0;                     // [WARPS][ring]; later slot 1
    static constexpr int first_off = WARPS * ring;         // [WARPS][slot]: slot 0
    static constexpr int bars_off = first_off + WARPS * slot;
    static constexpr int bytes = bars_off + WARPS * S * 8;
    static_assert(bytes <= kAttnSmem, "two CTAs fit on an SM");
    static_assert(rec % 16 == 0 && slot % 16 == 0, "bulk copies and slots are 16-byte aligned");
};

struct Part {                          // a warp's partial result of an item
    int64_t item_begin, item_end;      // units; item_end = 0: none
    int64_t b;
    int h, rt;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// fp16 pair c - Z of nibble 0 (1) of both halves; z1 = 1024 + Z, z2 = 64 + Z.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w, uint32_t z1) {
    return f16x2_sub(dev::and_or<0x000F000Fu>(w, 0x64006400u), z1);
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w, uint32_t z2) {
    return f16x2_sub(dev::and_or<0x00F000F0u>(w, 0x54005400u), z2);
}
// Transpose of an 8 x 8 matrix of 16-bit values held as an MMA fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar) : "memory");
}

// Where row `row` of a sequence (head h of the key heads) lies: its token,
// or -1 when the row does not exist or its token is not among the T.
__device__ __forceinline__ int64_t row_token(int64_t row, int64_t n, int share, int64_t cu0,
                                             int64_t T) {
    if (row >= n * share) return -1;
    const int64_t tok = cu0 + row / share;
    return tok >= 0 && tok < T ? tok : -1;
}

// What a row's sums are multiplied with at the end: 2^(nm - m) / l; 0 for a
// row that saw no key, NaN when l is.
__device__ __forceinline__ float row_factor(float m, float nm, float l) {
    return l > 0.0f ? ex2(nm - m) / l : l;
}

// Adds the `count` partial results part(0), part(1), ... of an item in that
// order, all threads of the CTA: into the partial result `dst` when it is not
// null, else normalised into the output.
template <int D, int NB, bool GLOBAL, typename F>
__device__ __forceinline__ void merge_parts(const AttnArgs &p, F part, int count, float *dst,
                                            const Part &it, int tid, int threads) {
    using L = Slot<D, NB>;
    const int64_t cu0 = p.cu[it.b], n = (int64_t)p.cu[it.b + 1] - cu0;
    auto ld = [](const float *q) { return GLOBAL ? __ldcg(q) : *q; };
    for (int e = tid; e < L::R * D; e += threads) {
        const int row = e / D, d = e - row * D;
        float m = kNoMax, nm = kNoMax;
        for (int i = 0; i < count; ++i) {
            const float *s = part(i) + L::stats + row;
            m = fmaxf(m, ld(s));
            nm = fmaxf(nm, ld(s + L::R));
        }
        float l = 0.0f, o = 0.0f;
        for (int i = 0; i < count; ++i) {
            const float *q = part(i), *s = q + L::stats + row;
            l += ld(s + 2 * L::R) * ex2(ld(s) - m);
            o += ld(q + row * L::pitch + d) * ex2(ld(s + L::R) - nm);
        }
        if (dst) {
            __stcg(dst + row * L::pitch + d, o);
            if (d == 0) {
                __stcg(dst + L::stats + row, m);
                __stcg(dst + L::stats + L::R + row, nm);
                __stcg(dst + L::stats + 2 * L::R + row, l);
            }
        } else {
            const int64_t r = (int64_t)it.rt * L::R + row;
            const int64_t tok = row_token(r, n, p.share, cu0, p.T);
            if (tok >= 0)
                p.out[tok * p.out_stride + ((int64_t)it.h * p.share + r % p.share) * D + d] =
                    (uint16_t)dev::f32_to_bf16_rne(o * row_factor(m, nm, l));
        }
    }
}

template <int D, int G, int NB, int WARPS, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) kv4_attention_kernel(const AttnArgs p) {
    using L = AttnLayout<D, G, NB, WARPS>;
    using SL = Slot<D, NB>;
    constexpr int NG = L::NG, S = L::S, R = 8 * NB, kThreads = 32 * WARPS;
    constexpr int KW = D / 32;                     // K words per token and lane; V words per lane and p
    constexpr int VW = D / 64;                     // 64-wide spans of d
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t pre[kThreads + 1];          // units before each thread's sequences
    __shared__ int64_t warp_sum[WARPS];
    __shared__ Part parts[2 * WARPS];
    __shared__ uint32_t abort_word;
    __shared__ int last_flag[2];
    volatile uint32_t *abort_flag = &abort_word;
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, tig = lane & 3;

    // ---- units of all sequences: every CTA adds them up itself ----
    const int64_t per = (p.B + kThreads - 1) / kThreads;       // sequences per thread
    int64_t mine = 0;
    for (int64_t i = 0; i < per; ++i) {
        const int64_t b = tid * per + i;
        if (b < p.B) {
            const int64_t len = p.kv_lens[b];
            if (blockIdx.x == 0 && (len < 0 || len > p.capacity)) atomicOr(p.err_word, kErrIndex);
            mine += seq_work(p.cu[b], p.cu[b + 1], len, p.capacity, p.window, p.share, p.kv_heads,
                             R).units;
        }
    }
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    if (tid < 2 * WARPS) parts[tid].item_end = 0;
    if (tid == 0) abort_word = 0u;
    if (lane == 0)
        for (int s = 0; s < S; ++s) mbar_init(sbase + L::bars_off + 8u * (warp * S + s), 1);
    if (tid == 0) asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    int64_t before = 0, units = 0;
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += warp_sum[w];
        units += warp_sum[w];
    }
    pre[tid + 1] = before + scan;
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const int64_t ctas = active_ctas(units, gridDim.x, p.min_units);
    if (units == 0 || blockIdx.x >= ctas) return;
    const int64_t cta_begin = range_begin(blockIdx.x, units, ctas);
    const int64_t cta_end = range_begin(blockIdx.x + 1, units, ctas);
    const int64_t w_begin = cta_begin + range_begin(warp, cta_end - cta_begin, WARPS);
    const int64_t w_end = cta_begin + range_begin(warp + 1, cta_end - cta_begin, WARPS);

    const uint32_t ring = sbase + L::ring_off + (uint32_t)warp * L::ring;
    const uint32_t bar0 = sbase + L::bars_off + 8u * (uint32_t)(warp * S);
    int stage = 0;                                 // next stage to consume
    uint32_t phase = 0;
    bool ok = true;
    int in_flight = 0;                             // copies to wait for after a failed wait

    if (w_begin < w_end) {
        // the sequence that holds unit w_begin
        int lo = 0;
        for (int i = lane; i < kThreads; i += 32)
            if (pre[i] <= w_begin) lo = i;
#pragma unroll
        for (int o = 16; o; o >>= 1) lo = max(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        // (threads without units share their prefix with the next one, so the
        // last thread at or below w_begin has units)
        int64_t b = lo * per, seq_begin = pre[lo];
        SeqWork sw;
        for (;; ++b) {
            sw = seq_work(p.cu[b], p.cu[b + 1], p.kv_lens[b], p.capacity, p.window, p.share,
                          p.kv_heads, R);
            if (w_begin < seq_begin + sw.units) break;
            seq_begin += sw.units;
        }
        int64_t u = w_begin;
        int64_t item = (u - seq_begin) / sw.blocks;            // (head, row tile) of the sequence
        while (u < w_end && ok) {
            while (u >= seq_begin + sw.units) {                // next sequence with units
                seq_begin += sw.units;
                ++b;
                sw = seq_work(p.cu[b], p.cu[b + 1], p.kv_lens[b], p.capacity, p.window, p.share,
                              p.kv_heads, R);
                item = 0;
            }
            const int h = (int)(item / sw.row_tiles), rt = (int)(item - h * sw.row_tiles);
            const int64_t item_begin = seq_begin + item * sw.blocks;
            const int64_t item_end = item_begin + sw.blocks;
            const int64_t seg_end = item_end < w_end ? item_end : w_end;
            const int64_t blk0 = sw.block0 + (u - item_begin);
            const int nblk = (int)(seg_end - u);
            const int64_t cu0 = p.cu[b];
            const int32_t *table = p.page_table + b * p.max_pages;

            // ---- copies: record of block i goes to stage (stage + i) % S ----
            int64_t rec_cur = 0;                   // lane i: record of block 32 * chunk + i
            uint32_t bad = 0;                      // stages whose block has no page
            const int stage0 = stage;
            auto load_chunk = [&](int first) {
                const int i = first + lane;
                rec_cur = -1;
                if (i < nblk && (blk0 + i) * kBlock < sw.len)
                    rec_cur = record_index(table, p.max_pages, p.num_pages, p.kv_heads, h,
                                           p.page_blocks, blk0 + i);
            };
            auto issue = [&](int i) {              // block i of the segment
                if ((i & 31) == 0) load_chunk(i);
                const int64_t rec = __shfl_sync(0xFFFFFFFFu, rec_cur, i & 31);
                int s = stage0 + i % S;
                if (s >= S) s -= S;
                bad = rec < 0 ? bad | (1u << s) : bad & ~(1u << s);
                if (lane == 0) {
                    if (rec < 0) {
                        mbar_arrive(bar0 + 8u * s);
                    } else {
                        mbar_arrive_expect_tx(bar0 + 8u * s, (uint32_t)L::rec);
                        bulk_copy(ring + (uint32_t)s * L::rec, p.cache + rec * L::rec,
                                  (uint32_t)L::rec, bar0 + 8u * s);
                    }
                }
            };
            for (int i = 0; i < S && i < nblk; ++i) issue(i);

            // ---- queries: B fragments, row gid of each 8-row tile ----
            uint32_t qf[NB][4 * KW];
            float kq[NB][2];                       // per column 2 tig, 2 tig + 1
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int64_t r = (int64_t)rt * R + 8 * nb + gid;
                const int64_t tok = row_token(r, sw.n, p.share, cu0, p.T);
                uint4 x[KW];
                const uint16_t *src =
                    p.q + tok * p.q_stride + ((int64_t)h * p.share + r % p.share) * D + 8 * tig;
                float big = 0.0f;
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    x[j] = tok >= 0 ? *reinterpret_cast<const uint4 *>(src + 32 * j)
                                    : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        big = fmaxf(big, fmaxf(fabsf(dev::bf16_lo(w[i])), fabsf(dev::bf16_hi(w[i]))));
                }
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                // 2^e brings the largest |q| into [2^14, 2^15) (e <= 126)
                const int be = (int)(__float_as_uint(big) >> 23);
                const int e = big > 0.0f ? min(14 + 127 - be, 126) : 0;
                const float f = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    float v[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] = dev::bf16_lo(w[i]) * f;
                        v[2 * i + 1] = dev::bf16_hi(w[i]) * f;
                    }
                    // a word's code pairs: nibbles (0,4), (1,5), (2,6), (3,7)
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[nb][4 * j + i] = pack_f16x2(v[i], v[i + 4]);
                }
                const float kr = p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
                kq[nb][0] = __shfl_sync(0xFFFFFFFFu, kr, 8 * tig);
                kq[nb][1] = __shfl_sync(0xFFFFFFFFu, kr, 8 * tig + 4);
            }
            // keys each column's row may see: [klo, khi)
            int64_t khi[NB][2], klo[NB][2];
            int64_t all_hi = sw.len, all_lo = 0, any_hi = 0;
            {
                const int64_t pos0 = sw.len - sw.n;
                const int64_t r0 = (int64_t)rt * R;
                int64_t r1 = r0 + R - 1;
                if (r1 > sw.n * p.share - 1) r1 = sw.n * p.share - 1;
                all_hi = pos0 + r0 / p.share + 1;
                any_hi = pos0 + r1 / p.share + 1;
                all_lo = p.window > 0 ? any_hi - p.window : 0;
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        int64_t r = r0 + 8 * nb + 2 * tig + c;
                        if (r > r1) r = r1;
                        khi[nb][c] = pos0 + r / p.share + 1;
                        klo[nb][c] = p.window > 0 ? khi[nb][c] - p.window : 0;
                    }
            }

            // ---- main loop ----
            float acc[4 * VW][NB][4], l[NB][2], m[NB][2], nm[NB][2], cf[NB][2];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][nb][c] = 0.0f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    l[nb][c] = 0.0f;
                    m[nb][c] = nm[nb][c] = kNoMax;
                    cf[nb][c] = 1.0f;
                }
            }
            for (int i = 0; i < nblk; ++i) {
                ok = mbar_wait(bar0 + 8u * stage, phase, p.wait_limit, abort_flag, p.err_word);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) {
                    in_flight = min(S, nblk - i);
                    break;
                }
                const uint32_t st = ring + (uint32_t)stage * L::rec;
                const int64_t key0 = (blk0 + i) * kBlock;
                if (key0 < any_hi) {
                    if ((bad >> stage) & 1u) {
                        // a block of existing keys without a page
                        if (lane == 0 && key0 < sw.len) atomicOr(p.err_word, kErrIndex);
                    } else {
                        // -- scores: tokens gid and gid + 8, columns 2 tig, 2 tig + 1
                        float s[NB][4];
                        uint32_t kw[2][KW];
#pragma unroll
                        for (int q = 0; q < (2 * KW + 3) / 4; ++q) {
                            const uint4 v = lds128(st + k_codes_off() + (uint32_t)(q * 512 + lane * 16));
                            const uint32_t t[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x) kw[(4 * q + x) / KW][(4 * q + x) % KW] = t[x];
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[nb][c] = 0.0f;
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr) {
                            float t[NB][4];
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int c = 0; c < 4; ++c) t[nb][c] = 0.0f;
                            uint32_t z1[2], z2[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t z = lds_u8(st + k_zeros_off(D, NG) + 16u * gr + gid + 8 * x);
                                z1[x] = (0x6400u + z) * 0x00010001u;
                                z2[x] = (0x5400u + 16u * z) * 0x00010001u;
                            }
#pragma unroll
                            for (int jj = 0; jj < G / 32; ++jj) {
                                const int j = gr * (G / 32) + jj;
#pragma unroll
                                for (int half = 0; half < 2; ++half) {
                                    const uint32_t a = kw[0][j] >> (8 * half), c = kw[1][j] >> (8 * half);
                                    const uint32_t a0 = codes_lo(a, z1[0]), a1 = codes_lo(c, z1[1]);
                                    const uint32_t a2 = codes_hi(a, z2[0]), a3 = codes_hi(c, z2[1]);
#pragma unroll
                                    for (int nb = 0; nb < NB; ++nb)
                                        mma_f16(t[nb], a0, a1, a2, a3, qf[nb][4 * j + 2 * half],
                                                qf[nb][4 * j + 2 * half + 1]);
                                }
                            }
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float sc = __uint_as_float(
                                    lds_u16(st + k_scales_off(D) + 32u * gr + 2u * (gid + 8 * x)) << 16);
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
                                        s[nb][2 * x + c] = fmaf(t[nb][2 * x + c], sc, s[nb][2 * x + c]);
                            }
                        }
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[nb][c] *= kq[nb][c & 1];
                        // -- V scales; binade of the largest
                        float vs[NG][2], ve[2];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t top = 0;
#pragma unroll
                            for (int gr = 0; gr < NG; ++gr) {
                                const uint32_t bits = lds_u16(st + v_scales_off(D, NG) + 32u * gr + 2u * (gid + 8 * x));
                                vs[gr][x] = __uint_as_float(bits << 16);
                                top = max(top, bits);
                            }
                            ve[x] = (float)((int)max(top >> 7, 1u) - 126);     // S < 2^ve
                        }
                        // -- masks
                        if (key0 < all_lo || key0 + kBlock > all_hi) {
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int64_t key = key0 + gid + 8 * x;
                                if (key >= sw.len) {       // never written: whatever it holds
#pragma unroll
                                    for (int gr = 0; gr < NG; ++gr) vs[gr][x] = 0.0f;
                                }
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
                                        if (key >= khi[nb][c] || key < klo[nb][c])
                                            s[nb][2 * x + c] = __int_as_float(0xFF800000);
                            }
                        }
                        // -- running maxima: raised only when a score is 2^8, or a
                        //    weight 2^4, above them (fp16 holds weights below 2^16)
                        bool raise = false;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                raise |= s[nb][c] > m[nb][c & 1] + 8.0f ||
                                         s[nb][c] + ve[c >> 1] > nm[nb][c & 1] + 4.0f;
                        if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    float a = fmaxf(s[nb][c], s[nb][c + 2]);
                                    float d = fmaxf(s[nb][c] + ve[0], s[nb][c + 2] + ve[1]);
#pragma unroll
                                    for (int o = 4; o < 32; o <<= 1) {
                                        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
                                        d = fmaxf(d, __shfl_xor_sync(0xFFFFFFFFu, d, o));
                                    }
                                    a = fmaxf(a, m[nb][c]);
                                    d = fmaxf(d, nm[nb][c]);
                                    const float fl = ex2(m[nb][c] - a), fo = ex2(nm[nb][c] - d);
                                    m[nb][c] = a;
                                    nm[nb][c] = d;
                                    cf[nb][c] = ex2(a - d);
                                    l[nb][c] *= fl;
#pragma unroll
                                    for (int y = 0; y < 4 * VW; ++y) {
                                        acc[y][nb][c] *= fo;
                                        acc[y][nb][c + 2] *= fo;
                                    }
                                }
                        }
                        // -- weights
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                s[nb][c] = ex2(s[nb][c] - m[nb][c & 1]);
                                l[nb][c & 1] += s[nb][c];
                                s[nb][c] *= cf[nb][c & 1];
                            }
                        uint32_t wf[NG][NB][2];
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    wf[gr][nb][x] = transpose8(pack_f16x2(
                                        s[nb][2 * x] * vs[gr][x], s[nb][2 * x + 1] * vs[gr][x]));
                        // -- values: rows d, columns 2 tig, 2 tig + 1
                        uint32_t vw[2][KW];
#pragma unroll
                        for (int q = 0; q < (2 * KW + 3) / 4; ++q) {
                            const uint4 v = lds128(st + v_codes_off(D) + (uint32_t)(q * 512 + lane * 16));
                            const uint32_t t[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x) vw[(4 * q + x) / KW][(4 * q + x) % KW] = t[x];
                        }
                        uint32_t z1[NG][2], z2[NG][2];     // tokens 8 p + 2 tig, + 1
#pragma unroll
                        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t z = dev::prmt(
                                    lds_u16(st + v_zeros_off(D, NG) + 16u * gr + 8u * x + 2u * tig), 0u, 0x4140u);
                                z1[gr][x] = z + 0x64006400u;
                                z2[gr][x] = 16u * z + 0x54005400u;
                            }
#pragma unroll
                        for (int wi = 0; wi < VW; ++wi)
#pragma unroll
                            for (int nib = 0; nib < 4; ++nib) {
                                const int gr = (64 * wi + 16 * nib) / G, sh = 8 * (nib >> 1);
                                const uint32_t w0 = vw[0][wi] >> sh, w1 = vw[0][VW + wi] >> sh;
                                const uint32_t w2 = vw[1][wi] >> sh, w3 = vw[1][VW + wi] >> sh;
                                uint32_t a0, a1, a2, a3;
                                if (nib & 1) {
                                    a0 = codes_hi(w0, z2[gr][0]); a1 = codes_hi(w1, z2[gr][0]);
                                    a2 = codes_hi(w2, z2[gr][1]); a3 = codes_hi(w3, z2[gr][1]);
                                } else {
                                    a0 = codes_lo(w0, z1[gr][0]); a1 = codes_lo(w1, z1[gr][0]);
                                    a2 = codes_lo(w2, z1[gr][1]); a3 = codes_lo(w3, z1[gr][1]);
                                }
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
                                    mma_f16(acc[4 * wi + nib][nb], a0, a1, a2, a3, wf[gr][nb][0],
                                            wf[gr][nb][1]);
                            }
                    }
                }
                // every register loaded from the stage has been consumed by an
                // MMA or a conversion: it may be filled again
                __syncwarp();
                if (++stage == S) { stage = 0; phase ^= 1u; }
                if (i + S < nblk) issue(i + S);
            }
            if (!ok) break;

            // ---- the segment's result ----
            const bool whole = u == item_begin && seg_end == item_end;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float t = l[nb][c];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
                    l[nb][c] = t;
                }
            float *slot = nullptr;
            if (!whole) {
                // the last segment's goes over the idle ring, an earlier one's
                // into the warp's own slot
                const bool last = seg_end == w_end;
                slot = reinterpret_cast<float *>(smem + (last ? L::ring_off + warp * L::ring
                                                              : L::first_off + warp * L::slot));
                if (lane == 0) {
                    Part &pt = parts[2 * warp + (last ? 1 : 0)];
                    pt.item_begin = item_begin;
                    pt.item_end = item_end;
                    pt.b = b;
                    pt.h = h;
                    pt.rt = rt;
                }
            }
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = 8 * nb + 2 * tig + c;
                    float f = 1.0f;
                    int64_t tok = -1;
                    uint16_t *dst = nullptr;
                    if (whole) {
                        const int64_t r = (int64_t)rt * R + row;
                        tok = row_token(r, sw.n, p.share, cu0, p.T);
                        f = row_factor(m[nb][c], nm[nb][c], l[nb][c]);
                        dst = p.out + tok * p.out_stride + ((int64_t)h * p.share + r % p.share) * D;
                    } else if (gid == 0) {
                        slot[SL::stats + row] = m[nb][c];
                        slot[SL::stats + R + row] = nm[nb][c];
                        slot[SL::stats + 2 * R + row] = l[nb][c];
                    }
#pragma unroll
                    for (int wi = 0; wi < VW; ++wi)
#pragma unroll
                        for (int nib = 0; nib < 4; ++nib)
#pragma unroll
                            for (int hi = 0; hi < 2; ++hi) {
                                const int d = 64 * wi + 16 * nib + 8 * hi + gid;
                                const float o = acc[4 * wi + nib][nb][2 * hi + c];
                                if (whole) {
                                    if (tok >= 0) dst[d] = (uint16_t)dev::f32_to_bf16_rne(o * f);
                                } else {
                                    slot[row * SL::pitch + d] = o;
                                }
                            }
                }
            u = seg_end;
            ++item;
        }
        if (!ok) {
            // a wait ran out: let the copies in flight land (bounded) before leaving
            for (int s = 0; s < in_flight; ++s) {
                mbar_drain(bar0 + 8u * stage, phase, p.err_word);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
        }
    }
    __syncthreads();
    if (*abort_flag) return;

    // ---- items shared by warps ----
    Part pend[2];                                   // items shared with other CTAs, by slot
    pend[0].item_end = pend[1].item_end = 0;
    auto slot_of = [&](int i) {                     // of parts[i]
        return reinterpret_cast<const float *>(
            smem + ((i & 1) ? L::ring_off + (i >> 1) * L::ring : L::first_off + (i >> 1) * L::slot));
    };
    for (int i = 0; i < 2 * WARPS;) {
        if (parts[i].item_end == 0) { ++i; continue; }
        const Part it = parts[i];
        const float *list[WARPS];                   // at most one part of an item per warp
        int count = 0;
        for (; i < 2 * WARPS; ++i) {
            if (parts[i].item_end == 0) continue;
            if (parts[i].item_begin != it.item_begin) break;
            list[count++] = slot_of(i);
        }
        float *dst = nullptr;
        if (it.item_begin < cta_begin || it.item_end > cta_end) {
            const int sl = partial_slot(it.item_begin, cta_begin);
            dst = p.partials + ((int64_t)blockIdx.x * 2 + sl) * SL::floats;
            pend[sl] = it;
        }
        merge_parts<D, NB, false>(p, [&](int x) { return list[x]; }, count, dst, it, tid, kThreads);
    }
    if (pend[0].item_end == 0 && pend[1].item_end == 0) return;
    // ---- items shared by CTAs: the last to arrive adds the parts in order ----
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        for (int sl = 0; sl < 2; ++sl) {
            last_flag[sl] = 0;
            if (pend[sl].item_end == 0) continue;
            const int64_t c0 = worker_of(pend[sl].item_begin, units, ctas);
            const int64_t c1 = worker_of(pend[sl].item_end - 1, units, ctas);
            last_flag[sl] = atomicAdd(&p.counters[c0], 1u) == (uint32_t)(c1 - c0);
        }
    }
    __syncthreads();
    for (int sl = 0; sl < 2; ++sl) {
        if (!last_flag[sl]) continue;
        __threadfence();
        const Part it = pend[sl];
        const int64_t c0 = worker_of(it.item_begin, units, ctas);
        const int64_t c1 = worker_of(it.item_end - 1, units, ctas);
        const int s0 = partial_slot(it.item_begin, range_begin(c0, units, ctas));
        const float *base = p.partials + 2 * c0 * SL::floats;
        merge_parts<D, NB, true>(
            p, [&](int x) { return base + ((int64_t)2 * x + (x == 0 ? s0 : 0)) * SL::floats; },
            (int)(c1 - c0 + 1), nullptr, it, tid, kThreads);
        if (tid == 0) p.counters[c0] = 0u;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// CTAs share an SM two by two; warps per CTA so that the accumulators and
// queries of NB 8-row tiles stay in registers.
template <int D, int NB>
constexpr int kAttnWarps = D == 256 ? (NB == 1 ? 4 : 3) : (NB == 1 ? 8 : 6);
constexpr int kAttnCtasPerSm = 2;

// Rows of a tile: 8 when a sequence has at most 8 rows per key head on
// average, else 16 (the keys are read once per tile).
int attn_tiles(int64_t T, int64_t B, int64_t share) { return T * share <= 8 * B ? 1 : 2; }

template <int D, int G, int NB>
qz_status launch_attn(const AttnArgs &args, int64_t ctas, cudaStream_t st) {
    constexpr int W = kAttnWarps<D, NB>;
    using L = AttnLayout<D, G, NB, W>;
    auto kernel = kv4_attention_kernel<D, G, NB, W, kAttnCtasPerSm>;
    static DeviceOnce attr_once;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return QZ_ERR_CUDA;
    }
    if (attr_once.run(dev, [&] {
            cudaError_t e = cudaFuncSetAttribute(
                kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            return e;
        }) != cudaSuccess)
        return QZ_ERR_CUDA;
    kernel<<<(unsigned)ctas, 32 * W, L::bytes, st>>>(args);
    return launch_status();
}

template <template <int, int> class Op, typename... A>
qz_status dispatch(int64_t D, int64_t G, A &&...a) {
    if (D == 64) return G == 32 ? Op<64, 32>::go(a...) : Op<64, 64>::go(a...);
    if (D == 128)
        return G == 32 ? Op<128, 32>::go(a...) : G == 64 ? Op<128, 64>::go(a...)
                                                         : Op<128, 128>::go(a...);
    return G == 64 ? Op<256, 64>::go(a...) : Op<256, 128>::go(a...);
}

template <int D, int G>
struct Append {
    static qz_status go(const StoreArgs &p, unsigned grid, cudaStream_t st) {
        kv4_append_kernel<D, G><<<grid, 32 * kStoreWarps, 0, st>>>(p);
        return launch_status();
    }
};
template <int D, int G>
struct Read {
    static qz_status go(const StoreArgs &p, unsigned grid, cudaStream_t st) {
        kv4_read_kernel<D, G><<<grid, 32 * kStoreWarps, 0, st>>>(p);
        return launch_status();
    }
};
template <int D, int G>
struct Attend {
    static qz_status go(const AttnArgs &p, int tiles, int64_t ctas, cudaStream_t st) {
        return tiles == 1 ? launch_attn<D, G, 1>(p, ctas, st) : launch_attn<D, G, 2>(p, ctas, st);
    }
};

StoreArgs store_args(const Kv4Cache &c) {
    StoreArgs p{};
    p.cache = static_cast<uint8_t *>(c.cache);
    p.page_table = static_cast<const int32_t *>(c.page_table);
    p.kv_lens = static_cast<const int32_t *>(c.kv_lens);
    p.cu = static_cast<const int32_t *>(c.cu);
    p.T = c.T; p.B = c.B;
    p.max_pages = c.max_pages; p.num_pages = c.num_pages;
    p.kv_heads = (int)c.kv_heads; p.page_size = (int)c.page_size;
    p.err_word = device_error_word();
    return p;
}

size_t slot_bytes(int64_t D, int tiles) { return (size_t)(8 * tiles * (D + 4) + 32 * tiles) * 4; }

}  // namespace

size_t kv4_record_bytes(int64_t D, int64_t G) { return (size_t)record_bytes(D, G); }

constexpr size_t kCounterBytes = (kSmCount * kAttnCtasPerSm * sizeof(uint32_t) + 255) & ~size_t(255);

// Two slots and a counter for every CTA that a device may run (both tile
// sizes, so that one buffer serves every call).
size_t kv4_attention_workspace_bytes(int64_t D) {
    return kCounterBytes + (size_t)kSmCount * kAttnCtasPerSm * 2 * slot_bytes(D, 2);
}

qz_status launch_kv4_append(const Kv4Cache &c, const void *k, const void *v, int64_t k_stride,
                            int64_t v_stride, cudaStream_t st) {
    StoreArgs p = store_args(c);
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    return dispatch<Append>(c.head_dim, c.group_size, p,
                            (unsigned)ceil_div(c.T * c.kv_heads, kStoreWarps), st);
}

qz_status launch_kv4_read(const Kv4Cache &c, void *k, void *v, cudaStream_t st) {
    StoreArgs p = store_args(c);
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    p.k_out = static_cast<uint16_t *>(k);
    p.v_out = static_cast<uint16_t *>(v);
    return dispatch<Read>(c.head_dim, c.group_size, p,
                          (unsigned)ceil_div(c.T * c.kv_heads, kStoreWarps), st);
}

qz_status launch_kv4_attention(const Kv4Cache &c, const void *q, int64_t q_stride, int64_t q_heads,
                               float scale, int64_t window, void *out, int64_t out_stride,
                               void *workspace, cudaStream_t st) {
    AttnArgs p{};
    p.q = static_cast<const uint16_t *>(q);
    p.q_stride = q_stride;
    p.cache = static_cast<const uint8_t *>(c.cache);
    p.page_table = static_cast<const int32_t *>(c.page_table);
    p.kv_lens = static_cast<const int32_t *>(c.kv_lens);
    p.cu = static_cast<const int32_t *>(c.cu);
    p.T = c.T; p.B = c.B;
    p.max_pages = c.max_pages; p.num_pages = c.num_pages;
    p.window = window;
    p.capacity = c.max_pages * c.page_size;
    p.kv_heads = (int)c.kv_heads;
    p.share = (int)(q_heads / c.kv_heads);
    p.page_blocks = (int)(c.page_size / kBlock);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.out = static_cast<uint16_t *>(out);
    p.out_stride = out_stride;
    const int tiles = attn_tiles(c.T, c.B, p.share);
    const int64_t ctas = (int64_t)device_sm_count() * kAttnCtasPerSm;
    // counters first: their place does not depend on the tile size
    p.counters = static_cast<uint32_t *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + kCounterBytes);
    p.min_units = 32;
    p.wait_limit = device_wait_limit();
    p.err_word = device_error_word();
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    return dispatch<Attend>(c.head_dim, c.group_size, p, tiles, ctas, st);
}

}  // namespace qz
