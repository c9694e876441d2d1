// qz_kv4.cu -- the paged 4-bit key/value cache: append (quantize), read
// (dequantize) and attention over it.
//
// The cache holds the int4 asymmetric group format of qz_quantize_pack per
// (token, head): codes c, a bf16 scale S and a zero-point Z per group of g of
// the head's D values, standing for S (c - Z).  Layout and work split:
// qz_kv4_index.cuh.
#include <cuda_runtime.h>

#include "qz_kv4_index.cuh"
#include "qz_serving.cuh"
#include "qz_sm100.cuh"

namespace qz {
namespace {

using namespace sm100;
using namespace kv4;

constexpr unsigned kErrIndex = 2u;     // bit of the device error word: bad page or position

// ---------------------------------------------------------------------------
// append and read
// ---------------------------------------------------------------------------
// A unit is one record's worth of tokens: 16 positions (or the part of them
// that is the call's) of one head.  A lane works on 64 consecutive values of
// one token ("chunk"), which hold whole groups (or half a group of 128) and
// whole 32-bit words of K and 16-bit units of V; a pass is 32 chunks.  Passes'
// values and the record go through the warp's shared memory, so that global
// memory is read and written in whole rows and whole records.  (With a warp per
// token and head and scattered stores, 8057 prompt tokens written and read back
// took 76 us instead of 35, cold; 8 key heads of 128.)
// Measured there, warm: append 14.0 us, read 10.0 us (42 MB each: 0.47 and 0.65
// of the 6449 GB/s of a copy); 35 thousand tokens read back cold 41 us (175 MB,
// 0.66), 45 us without the next unit's record under way.  The read issues on
// 0.37 of the cycles and waits mostly for loads (counters, before that
// prefetch): latency, not instructions.  The append issues on 0.45 with 12 warps
// active per SM, and waits mostly for loads too; fetching the next unit's rows
// to L2 or L1 first changed nothing (14.0 to 14.2 us), five CTAs per SM in place
// of four took 16.0.
struct StoreArgs {
    const uint16_t *k, *v;             // append: input
    uint16_t *k_out, *v_out;           // read: output
    int64_t k_stride, v_stride;        // elements between tokens
    uint8_t *cache;
    const int32_t *page_table, *kv_lens, *cu;
    int64_t max_pages, num_pages;
    int T, B, kv_heads, page_blocks;
    unsigned int *err_word;
};

constexpr int kStoreWarps = 4;
constexpr int kStoreThreads = 32 * kStoreWarps;
constexpr int kAppendCtas = 4;         // per SM: 128 registers per thread
template <int D>
constexpr int kReadCtas = D == 256 ? 4 : 5;        // per SM: 128 or 96 registers per thread
constexpr int kChunkPitch = 144;       // bytes of a staged chunk: 64 bf16, padded against bank conflicts

template <int D, int G>
struct StoreLayout {
    static constexpr int NG = D / G;
    static constexpr int chunks = D / 64;                   // of a token
    static constexpr int rec = (int)record_bytes(D, G);
    static constexpr int tile = 32 * kChunkPitch;           // the values of a pass
    static constexpr int per_warp = tile + rec;
    static_assert(rec >= 2 * D, "append_token's buffer");
    static_assert(kReadCtas<D> * (kStoreWarps * per_warp + 4096) <= 228 * 1024, "the CTAs fit on an SM");
};

// Chunk `id` (0 .. 32 chunks - 1) of a unit: keys, then values, token by token.
template <int D>
struct Chunk {
    int which, t, wi;
    __device__ __forceinline__ explicit Chunk(int id)
        : which(id / (16 * (D / 64))), t(id % (16 * (D / 64)) / (D / 64)), wi(id % (D / 64)) {}
};

// Adds up the sequences' units and finds where warp `gw` of `warps` starts:
// calls unit(b, work, index in the sequence) for each unit of its range.
template <typename F>
__device__ __forceinline__ void for_units(const StoreArgs &p, F unit) {
    __shared__ int64_t pre[kStoreThreads + 1], warp_sum[kStoreWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto work_of = [&](int b) {
        return store_work(p.cu[b], p.cu[b + 1], p.kv_lens[b], p.T, p.kv_heads);
    };
    const int per = (p.B + kStoreThreads - 1) / kStoreThreads;
    int64_t scan = 0;
    for (int i = 0; i < per; ++i)
        if (tid * per + i < p.B) scan += work_of(tid * per + i).units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) warp_sum[warp] = scan;
    __syncthreads();
    int64_t before = 0, units = 0;
#pragma unroll
    for (int w = 0; w < kStoreWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        units += warp_sum[w];
    }
    pre[tid + 1] = before + scan;
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const int64_t warps = (int64_t)gridDim.x * kStoreWarps;
    const int64_t quota = quotient(units + warps - 1, warps);
    // consecutive units go to different CTAs while there are few
    int64_t u = ((int64_t)warp * gridDim.x + blockIdx.x) * quota;
    const int64_t end = min(u + quota, units);
    if (u >= end) return;
    int lo = 0;
    for (int i = lane; i < kStoreThreads; i += 32)
        if (pre[i] <= u) lo = i;
    lo = __reduce_max_sync(0xFFFFFFFFu, lo);
    int b = lo * per;
    int64_t begin = pre[lo];
    StoreWork w = work_of(b);
    while (u < end) {
        while (u >= begin + w.units) {
            begin += w.units;
            w = work_of(++b);
        }
        unit(b, w, u - begin);
        ++u;
    }
}

// Codes of 8 values (word: value i in nibble i), clamp(round(x / S + Z)) as
// qz_quantize_pack forms them: with r = 1/S rounded, fma(x, r, Z + 192) lies on
// the same side of every half-way point as x / S + Z (bf16 x and S keep x / S +
// Z at least 2^-10 from a half-way point it does not hit; the argument is
// written out at chunk_codes in qz_quantize.cu), and adding 1.5 2^23 - 192
// rounds half to even into the low mantissa bits.  Two values per fma and add.
__device__ __forceinline__ uint32_t codes8(const uint4 &x, float r, float zc) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    uint32_t pair[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a, c;
        asm("{\n\t.reg .b64 xx, rr, zz, kk, yy;\n\t"
            "mov.b64 xx, {%2, %3};\n\tmov.b64 rr, {%4, %4};\n\t"
            "mov.b64 zz, {%5, %5};\n\tmov.b64 kk, {%6, %6};\n\t"
            "fma.rn.f32x2 yy, xx, rr, zz;\n\tadd.rn.f32x2 yy, yy, kk;\n\t"
            "mov.b64 {%0, %1}, yy;\n\t}"
            : "=r"(a), "=r"(c)
            : "r"(u[i] << 16), "r"(u[i] & 0xFFFF0000u), "r"(__float_as_uint(r)),
              "r"(__float_as_uint(zc)), "r"(__float_as_uint(12582912.0f - 192.0f)));
        a = min(a, 0x4B40000Fu);
        c = min(c, 0x4B40000Fu);
        pair[i] = dev::and_or<0x0Fu>(a, c << 4);            // byte 0: both codes
    }
    return dev::prmt(dev::prmt(pair[0], pair[1], 0x0040u), dev::prmt(pair[2], pair[3], 0x0040u),
                     0x5410u);
}
// The same with the IEEE division, for scales whose inverse overflows.
__device__ __forceinline__ uint32_t code4_exact(float x, float s, float z) {
    const int q = (int)rintf(__fadd_rn(__fdiv_rn(x, s), z));
    return (uint32_t)min(max(q, 0), 15);
}
__device__ __noinline__ uint32_t codes8_exact(uint4 x, float s, float z) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        word |= code4_exact(dev::bf16_lo(u[i]), s, z) << (8 * i) |
                code4_exact(dev::bf16_hi(u[i]), s, z) << (8 * i + 4);
    return word;
}

// One value as codes8 (or, where the inverse overflows, codes8_exact) forms it,
// values that are not finite included.
__device__ __forceinline__ uint32_t code4(float x, float s, float inv, float z) {
    if (!(inv < __int_as_float(0x7F800000))) return code4_exact(x, s, z);
    const float y = __fadd_rn(__fmaf_rn(x, inv, __fadd_rn(z, 192.0f)), 12582912.0f - 192.0f);
    return min(__float_as_uint(y), 0x4B40000Fu) & 0x0Fu;
}

// Transposes 4 x 8 nibbles: words a, b, c, d of 8 nibbles -> units g = 0..7 of
// four nibbles (a_g, b_g, c_g, d_g); out[0] = units 0, 2, out[1] = 4, 6,
// out[2] = 1, 3, out[3] = 5, 7 (low half, high half).
__device__ __forceinline__ void nibbles_to_units(uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                                 uint32_t (&out)[4]) {
    constexpr uint32_t m = 0x0F0F0F0Fu;
    const uint32_t e0 = (a & m) | ((b & m) << 4), e1 = ((a >> 4) & m) | (b & ~m);
    const uint32_t f0 = (c & m) | ((d & m) << 4), f1 = ((c >> 4) & m) | (d & ~m);
    out[0] = dev::prmt(e0, f0, 0x5140u);
    out[1] = dev::prmt(e0, f0, 0x7362u);
    out[2] = dev::prmt(e1, f1, 0x5140u);
    out[3] = dev::prmt(e1, f1, 0x7362u);
}
// The inverse: units u[0..7] (low halves) -> words a, b, c, d.
__device__ __forceinline__ void units_to_nibbles(const uint32_t (&u)[8], uint32_t &a, uint32_t &b,
                                                 uint32_t &c, uint32_t &d) {
    constexpr uint32_t m = 0x0F0F0F0Fu;
    const uint32_t p0 = dev::prmt(u[0], u[2], 0x5140u), p1 = dev::prmt(u[4], u[6], 0x5140u);
    const uint32_t q0 = dev::prmt(u[1], u[3], 0x5140u), q1 = dev::prmt(u[5], u[7], 0x5140u);
    const uint32_t e0 = dev::prmt(p0, p1, 0x5410u), f0 = dev::prmt(p0, p1, 0x7632u);
    const uint32_t e1 = dev::prmt(q0, q1, 0x5410u), f1 = dev::prmt(q0, q1, 0x7632u);
    a = (e0 & m) | ((e1 & m) << 4);
    b = ((e0 >> 4) & m) | (e1 & ~m);
    c = (f0 & m) | ((f1 & m) << 4);
    d = ((f0 >> 4) & m) | (f1 & ~m);
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Scale (bf16 bits) and zero of a group with the 0-extended range [lo, hi]
// (qz.h: S = (max - min) / 15 in fp32 stored as bf16 rounded up, 0 -> 1).
__device__ __forceinline__ uint32_t group_scale(float lo, float hi, float &s, float &z) {
    s = __fdiv_rn(__fsub_rn(hi, lo), 15.0f);
    if (s == 0.0f) s = 1.0f;
    const uint32_t sb = dev::bf16_round_up_bits(s);
    s = __uint_as_float(sb << 16);
    z = (float)(int)-rintf(__fdiv_rn(lo, s));      // 0 for a NaN
    return sb;
}

// One token of one head into its record `dst`; a lane holds D / 32 consecutive
// values of the keys, then of the values.  `buf`: 2 D bytes of the warp's own.
template <int D, int G>
__device__ __forceinline__ void append_token(const uint16_t *k, const uint16_t *v, int t, uint8_t *dst,
                                             uint8_t *buf, int lane) {
    constexpr int NG = D / G, V = D / 32, LPG = G / V;       // LPG lanes per group
    uint32_t w[2][V / 2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(which ? v : k) + lane * (V / 2);
        if constexpr (V == 2) {
            w[which][0] = __ldg(src);
        } else if constexpr (V == 4) {
            const uint2 x = __ldg(reinterpret_cast<const uint2 *>(src));
            w[which][0] = x.x; w[which][1] = x.y;
        } else {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src));
            w[which][0] = x.x; w[which][1] = x.y; w[which][2] = x.z; w[which][3] = x.w;
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float mn = 0.0f, mx = 0.0f;
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            mn = fminf(mn, fminf(dev::bf16_lo(w[which][i]), dev::bf16_hi(w[which][i])));
            mx = fmaxf(mx, fmaxf(dev::bf16_lo(w[which][i]), dev::bf16_hi(w[which][i])));
        }
#pragma unroll
        for (int o = 1; o < LPG; o <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        }
        float s, z;
        const uint32_t sb = group_scale(mn, mx, s, z);
        const float inv = __frcp_rn(s);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            buf[which * D + lane * V + 2 * i] = (uint8_t)code4(dev::bf16_lo(w[which][i]), s, inv, z);
            buf[which * D + lane * V + 2 * i + 1] =
                (uint8_t)code4(dev::bf16_hi(w[which][i]), s, inv, z);
        }
        if ((lane & (LPG - 1)) == 0) {
            const int so = 16 * (lane / LPG) + t;
            *reinterpret_cast<uint16_t *>(dst + (which ? v_scales_off(D, NG) : k_scales_off(D)) +
                                          2 * so) = (uint16_t)sb;
            dst[(which ? v_zeros_off(D, NG) : k_zeros_off(D, NG)) + so] = (uint8_t)(int)z;
        }
    }
    __syncwarp();
    if (lane < D / 8) {
        const uint2 x = reinterpret_cast<const uint2 *>(buf)[lane];
        const uint32_t lo = x.x | (x.x >> 4), hi = x.y | (x.y >> 4);   // pairs in bytes 0 and 2
        *reinterpret_cast<uint32_t *>(dst + k_codes_off() + k_word_byte(D, t, lane)) =
            dev::prmt(lo, hi, 0x6420u);
    }
    for (int u = lane; u < D / 4; u += 32) {
        const int gid = u & 7, hi = (u >> 3) & 1, wi = u >> 4;
        uint32_t x = 0;
#pragma unroll
        for (int n = 0; n < 4; ++n) x |= (uint32_t)buf[D + 64 * wi + 16 * n + 8 * hi + gid] << (4 * n);
        *reinterpret_cast<uint16_t *>(dst + v_codes_off(D) + v_unit_byte(D, t, wi, hi, gid)) =
            (uint16_t)x;
    }
    __syncwarp();
}

template <int D, int G>
__global__ void __launch_bounds__(kStoreThreads, kAppendCtas) kv4_append_kernel(const StoreArgs p) {
    using L = StoreLayout<D, G>;
    constexpr int NG = L::NG, CH = L::chunks, W8 = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31;
    uint8_t *tile = smem + (threadIdx.x >> 5) * L::per_warp, *rec = tile + L::tile;
    for_units(p, [&](int b, const StoreWork &w, int64_t index) {
        const int i = (int)quotient(index, p.kv_heads), h = (int)(index - (int64_t)i * p.kv_heads);
        const int block = w.block0 + i;
        const int lo = block_lo(w, block), hi = block_hi(w, block);
        const int64_t r = record_index(p.page_table + (int64_t)b * p.max_pages, p.max_pages,
                                       p.num_pages, p.kv_heads, h, p.page_blocks, block);
        if (r < 0) {
            if (lane == 0) atomicOr(p.err_word, kErrIndex);
            return;
        }
        const int64_t row0 = p.cu[b] + ((int64_t)block * kBlock - w.first);   // of token 0
        uint8_t *dst = p.cache + r * L::rec;
        const int end = (int)min((int64_t)hi, p.T - row0);
        // few tokens, as in decoding: one at a time, all lanes on it (one new
        // token of each of 32 sequences 3.9 us, by the passes below 6.4)
        if (end - lo <= 2) {
            // ---- a token or two (decoding): a lane takes D / 32 values ----
            for (int t = lo; t < end; ++t)
                append_token<D, G>(p.k + (row0 + t) * p.k_stride + (int64_t)h * D,
                                   p.v + (row0 + t) * p.v_stride + (int64_t)h * D, t, dst, rec, lane);
            return;
        }
        // a pass's values, 16 bytes per lane and load
        uint4 v[8];
        auto load = [&](int pass) {
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const Chunk<D> c(32 * pass + 4 * x + lane / 8);
                v[x] = c.t >= lo && c.t < end
                           ? __ldg(reinterpret_cast<const uint4 *>(
                                 (c.which ? p.v : p.k) + (int64_t)h * D +
                                 (row0 + c.t) * (c.which ? p.v_stride : p.k_stride) + 64 * c.wi +
                                 8 * (lane % 8)))
                           : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        load(0);
#pragma unroll
        for (int pass = 0; pass < CH; ++pass) {
#pragma unroll
            for (int x = 0; x < 8; ++x)
                *reinterpret_cast<uint4 *>(tile + (4 * x + lane / 8) * kChunkPitch + 16 * (lane % 8)) = v[x];
            __syncwarp();
            if (pass + 1 < CH) load(pass + 1);
            const Chunk<D> ch(32 * pass + lane);
            const int which = ch.which, t = ch.t, wi = ch.wi;
            const uint8_t *src = tile + lane * kChunkPitch;
            uint4 x[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = *reinterpret_cast<const uint4 *>(src + 16 * q);
            constexpr int GC = G < 64 ? 64 / G : 1;         // groups of a chunk
            uint32_t codes[8];                              // word q: d = 8 q .. 8 q + 7
#pragma unroll
            for (int gc = 0; gc < GC; ++gc) {
                uint32_t mn2 = 0, mx2 = 0;                  // pairs, from 0
#pragma unroll
                for (int q = gc * (8 / GC); q < (gc + 1) * (8 / GC); ++q) {
                    mn2 = min_bf16x2(mn2, min_bf16x2(min_bf16x2(x[q].x, x[q].y), min_bf16x2(x[q].z, x[q].w)));
                    mx2 = max_bf16x2(mx2, max_bf16x2(max_bf16x2(x[q].x, x[q].y), max_bf16x2(x[q].z, x[q].w)));
                }
                float mn = fminf(dev::bf16_lo(mn2), dev::bf16_hi(mn2));
                float mx = fmaxf(dev::bf16_lo(mx2), dev::bf16_hi(mx2));
                if constexpr (G == 128) {
                    mn = fminf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                }
                float s, z;
                const uint32_t sb = group_scale(mn, mx, s, z);
                const float inv = __frcp_rn(s), zc = __fadd_rn(z, 192.0f);
                if (inv < __int_as_float(0x7F800000)) {
#pragma unroll
                    for (int q = gc * (8 / GC); q < (gc + 1) * (8 / GC); ++q)
                        codes[q] = codes8(x[q], inv, zc);
                } else {
#pragma unroll
                    for (int q = gc * (8 / GC); q < (gc + 1) * (8 / GC); ++q)
                        codes[q] = codes8_exact(x[q], s, z);
                }
                const int so = 16 * (G == 128 ? wi >> 1 : wi * GC + gc) + t;
                if (G != 128 || (wi & 1) == 0) {
                    *reinterpret_cast<uint16_t *>(
                        rec + (which ? v_scales_off(D, NG) : k_scales_off(D)) + 2 * so) = (uint16_t)sb;
                    rec[(which ? v_zeros_off(D, NG) : k_zeros_off(D, NG)) + so] = (uint8_t)(int)z;
                }
            }
            if (which == 0) {
                // words 2 wi and 2 wi + 1 of each lane slot c are neighbours
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint2 *>(rec + k_word_byte(D, t, 8 * wi + c)) =
                        make_uint2(codes[c], codes[4 + c]);
            } else {
                // unit (uh, g): codes d = 16 n + 8 uh + g, n = 0..3
#pragma unroll
                for (int uh = 0; uh < 2; ++uh) {
                    uint32_t u[4];
                    nibbles_to_units(codes[uh], codes[2 + uh], codes[4 + uh], codes[6 + uh], u);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int g8 = 4 * (y & 1) + (y >> 1);         // and g8 + 2
                        *reinterpret_cast<uint16_t *>(rec + v_codes_off(D) +
                                                      v_unit_byte(D, t, wi, uh, g8)) = (uint16_t)u[y];
                        *reinterpret_cast<uint16_t *>(rec + v_codes_off(D) +
                                                      v_unit_byte(D, t, wi, uh, g8 + 2)) =
                            (uint16_t)(u[y] >> 16);
                    }
                }
            }
            __syncwarp();
        }
        // ---- out: the whole record, or the bytes of the call's tokens alone ----
        if (lo == 0 && end == kBlock) {
            for (int e = lane; e < L::rec / 16; e += 32)
                reinterpret_cast<uint4 *>(dst)[e] = reinterpret_cast<const uint4 *>(rec)[e];
        } else {
            for (int e = lane; e < 16 * W8; e += 32) {
                const int t = e / W8, o = k_word_byte(D, t, e % W8);
                if (t >= lo && t < end)
                    *reinterpret_cast<uint32_t *>(dst + o) = *reinterpret_cast<uint32_t *>(rec + o);
            }
            for (int e = lane; e < 16 * (D / 4); e += 32) {
                const int t = e / (D / 4), u = e % (D / 4);
                const int o = v_codes_off(D) + v_unit_byte(D, t, u >> 4, (u >> 3) & 1, u & 7);
                if (t >= lo && t < end)
                    *reinterpret_cast<uint16_t *>(dst + o) = *reinterpret_cast<uint16_t *>(rec + o);
            }
            for (int e = lane; e < 2 * NG * 16; e += 32) {   // K groups, then V groups
                const int t = e & 15;
                if (t < lo || t >= end) continue;
                const int o = k_scales_off(D) + 2 * e, oz = k_zeros_off(D, NG) + e;
                *reinterpret_cast<uint16_t *>(dst + o) = *reinterpret_cast<uint16_t *>(rec + o);
                dst[oz] = rec[oz];
            }
        }
        __syncwarp();
    });
}

template <int D, int G>
__global__ void __launch_bounds__(kStoreThreads, kReadCtas<D>) kv4_read_kernel(const StoreArgs p) {
    using L = StoreLayout<D, G>;
    constexpr int NG = L::NG, CH = L::chunks, NV = L::rec / 16, VL = (NV + 31) / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31;
    uint8_t *tile = smem + (threadIdx.x >> 5) * L::per_warp, *rec = tile + L::tile;
    // a unit's record is loaded while the unit before it is worked on
    struct Unit {
        int64_t row0;                                       // output row of token 0
        int lo, hi, h;
        bool ok;                                            // its page exists
    };
    auto give = [&](const Unit &u, const uint4 (&v)[VL]) {
        const int64_t row0 = u.row0;
        const int lo = u.lo, hi = u.hi, h = u.h;
#pragma unroll
        for (int x = 0; x < VL; ++x)
            if (x * 32 + lane < NV) reinterpret_cast<uint4 *>(rec)[x * 32 + lane] = v[x];
        __syncwarp();
#pragma unroll
        for (int pass = 0; pass < CH; ++pass) {
            const Chunk<D> ch(32 * pass + lane);
            const int which = ch.which, t = ch.t, wi = ch.wi;
            uint32_t codes[8];                              // word q: d = 8 q .. 8 q + 7
            if (which == 0) {
                // words 2 wi and 2 wi + 1 of each lane slot c are neighbours
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint2 x = *reinterpret_cast<const uint2 *>(rec + k_word_byte(D, t, 8 * wi + c));
                    codes[c] = x.x;
                    codes[4 + c] = x.y;
                }
            } else {
#pragma unroll
                for (int uh = 0; uh < 2; ++uh) {
                    uint32_t u[8];
#pragma unroll
                    for (int g8 = 0; g8 < 8; ++g8)
                        u[g8] = *reinterpret_cast<const uint16_t *>(
                            rec + v_codes_off(D) + v_unit_byte(D, t, wi, uh, g8));
                    units_to_nibbles(u, codes[uh], codes[2 + uh], codes[4 + uh], codes[6 + uh]);
                }
            }
            uint8_t *dst = tile + lane * kChunkPitch;
            constexpr int GC = G < 64 ? 64 / G : 1;         // groups of a chunk
#pragma unroll
            for (int gc = 0; gc < GC; ++gc) {
                const int so = 16 * ((64 * wi + (64 / GC) * gc) / G) + t;
                uint32_t s2 = *reinterpret_cast<const uint16_t *>(
                    rec + (which ? v_scales_off(D, NG) : k_scales_off(D)) + 2 * so);
                uint32_t z2 = rec[(which ? v_zeros_off(D, NG) : k_zeros_off(D, NG)) + so];
                if (!u.ok) s2 = z2 = 0;
                s2 *= 0x00010001u;                          // (S, S)
                z2 = (0x4300u + z2) * 0x00010001u;          // bf16(128 + Z) twice
#pragma unroll
                for (int q = gc * (8 / GC); q < (gc + 1) * (8 / GC); ++q) {
                    uint32_t o[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)             // bf16(S (q - Z)), rounded once
                        o[y] = dequant_pair_nat(codes[q], codes[q] >> 4, y, s2, z2);
                    *reinterpret_cast<uint4 *>(dst + 16 * q) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const Chunk<D> c(32 * pass + 4 * x + lane / 8);
                const int64_t row = row0 + c.t;
                if (c.t >= lo && c.t < hi && row < p.T)
                    *reinterpret_cast<uint4 *>((c.which ? p.v_out : p.k_out) +
                                               (row * p.kv_heads + h) * D + 64 * c.wi + 8 * (lane % 8)) =
                        *reinterpret_cast<const uint4 *>(tile + (4 * x + lane / 8) * kChunkPitch +
                                                         16 * (lane % 8));
            }
            __syncwarp();
        }
    };
    Unit last{};
    last.h = -1;
    uint4 held[VL];
    for_units(p, [&](int b, const StoreWork &w, int64_t index) {
        const int i = (int)quotient(index, p.kv_heads), block = w.block0 + i;
        Unit u;
        u.h = (int)(index - (int64_t)i * p.kv_heads);
        u.lo = block_lo(w, block);
        u.hi = block_hi(w, block);
        u.row0 = p.cu[b] + ((int64_t)block * kBlock - w.first);
        const int64_t r = record_index(p.page_table + (int64_t)b * p.max_pages, p.max_pages,
                                       p.num_pages, p.kv_heads, u.h, p.page_blocks, block);
        u.ok = r >= 0;
        uint4 v[VL] = {};
        if (u.ok) {
            const uint4 *src = reinterpret_cast<const uint4 *>(p.cache + r * L::rec);
#pragma unroll
            for (int x = 0; x < VL; ++x)
                if (x * 32 + lane < NV) v[x] = __ldg(src + x * 32 + lane);
        } else if (lane == 0) {
            atomicOr(p.err_word, kErrIndex);
        }
        if (last.h >= 0) give(last, held);
        last = u;
#pragma unroll
        for (int x = 0; x < VL; ++x) held[x] = v[x];
    });
    if (last.h >= 0) give(last, held);
}

// ---------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------
// Row i of a sequence with n queries and len keys stands at position
// p = len - n + i and sees keys j <= p (and j > p - window):
//   s_j = scale sum_d q_d S_j (c_jd - Z_j),  P = softmax(s),
//   out_d = sum_j P_j S_j (c_jd - Z_j).
// Scores are integer products: a row's query is a 16-bit fixed-point number
// relative to its largest value (q = i 2^-e, |i| < 2^15: at most 2^-15 of that
// value off; bf16 values down to 2^-7 of it are exact), split into a signed
// high and an unsigned low byte, and the codes are the bytes of a word ANDed
// with 0x0F0F0F0F, and shifted by 4: 3 instructions for 8 codes, two mma.sync
// m16n8k32 with exact 32-bit sums.  Z and S stay out of the product:
//   sum_d q_d S (c - Z) = S 2^-e (sum_d i_d c - Z sum_d i_d).
// (As fp16 products with c - Z formed per code, the scores took 9 instructions
// for 8 codes.)
// For the values the codes enter the tensor cores as the exact fp16 integers
// c - Z.  Of a 16-bit half, nibble 0 ORed under fp16 1024 is 1024 + c and
// nibble 1 under 64 is 64 + c (one LOP3 each for the same nibble of both
// halves), and one packed subtraction of 1024 + Z or 64 + Z leaves c - Z; a
// shift by 8 does the other two.  (Leaving the subtraction out -- codes as fp16
// subnormals, Z taken off the sums -- saves 4 instructions per word, but the
// tensor core aligns a subnormal's products by its nominal exponent and loses
// their low bits: 2^-15 of the largest product, seen where one key holds the
// weight and c = Z.)
// The weights P_j S_j are rounded once to fp16 (2^-11 of each) for the second
// product: w_j = 2^(s_j - m) S_j 2^-E, m a row's running maximum of s_j (in
// powers of two) and E an exponent per row and group of channels that keeps the
// largest weight near 1 whatever the sizes of V (one for all rows of a warp would
// round a row by values that only other rows see, one for all groups a group by
// another's scales).  They move only when a weight reaches 2^12 (fp16 holds those
// below 2^16) or the weights of a step 2^100.  A group of zeros, which is stored
// with S = 1, adds nothing and sets no E: it is looked for when E would move.  The
// softmax's sum l of 2^(s_j - m) is fp32.
//
// Work.  Warps work alone: a warp takes a contiguous range of (head, block)
// units, keeps records of 16 tokens in a ring of its own (two per stage, one
// bulk copy each) and its sums in registers, 8 NB query rows as the columns
// of the tensor-core tiles (tokens x heads for the scores, d x heads for the
// result, so that the probabilities only need an 8 x 8 transpose between the
// two).  An item cut by warps is joined in shared memory, one cut by CTAs in
// the workspace by the last to arrive, parts added in order.
//
// Measured, 8 key heads of 128: 128 sequences of 1000..16000 tokens (785 MB, 32
// query heads) 165 us warm, 180 cold: 0.68 of the copy bandwidth; one sequence of
// 131001 tokens (64 query heads, two scales per head, 147 MB) 49 us warm, one of 777
// tokens 11 us.  A record of 16 tokens costs 262 warp instructions, 108 of them
// integer and logic, 94 on the multiply pipes, 16 loads and stores, 16 tensor
// products.  At 32 sequences the schedulers issue on 0.53 of the cycles, the ALU pipe
// is busy for 0.43 and the tensor pipe for 0.23 of them, and the three warps of a
// scheduler wait mostly for the results of earlier instructions: latency of
// dependent instructions, no unit that is full.  From 8 to 32 sequences the records
// stream at 0.81 of the copy bandwidth, and 20 us a call do not depend on the length.
// Keys whose group is all zeros cost a search each step while nothing else has been
// seen (64 x 4000 tokens, the last of four groups zero: 93 us, 134).
struct AttnArgs {
    const uint16_t *q;
    int64_t q_stride;                  // elements between tokens
    const uint8_t *cache;
    const int32_t *page_table, *kv_lens, *cu;
    int64_t max_pages, num_pages;
    int T, B, window, capacity, kv_heads, share, page_blocks;
    float scale_log2;                  // scale * log2(e)
    uint16_t *out;
    int64_t out_stride;
    float *partials;                   // [ctas][2][Slot]
    uint32_t *counters;                // [ctas]
    int min_units, whole_units;        // see cta_quota
    uint64_t wait_limit;
    unsigned int *err_word;
};

constexpr float kNoMax = -3.4e38f;     // running maximum before any key

// A partial result of a row tile: [R][D + 4] fp32 sums, then m and l per row.
template <int D, int NB>
struct Slot {
    static constexpr int R = 8 * NB;
    static constexpr int pitch = D + 4;                    // floats: rows 8 apart in banks
    static constexpr int stats = R * pitch;                // m[R], l[R]
    static constexpr int floats = R * pitch + 2 * R;
    static constexpr int bytes = floats * 4;
};

// Dynamic shared memory of a CTA: 228 KB per SM, 1 KB of it reserved per CTA,
// and up to 5 KB of static arrays.
constexpr int attn_smem(int ctas) { return (ctas == 2 ? 108 : 221) * 1024; }

template <int D, int G, int NB, int WARPS, int CTAS>
struct AttnLayout {
    static constexpr int NG = D / G;
    static constexpr int rec = (int)record_bytes(D, G);
    static constexpr int slot = Slot<D, NB>::bytes;
    static constexpr int ring_bytes(int s) {
        return ((2 * s * rec > slot ? 2 * s * rec : slot) + 15) & ~15;
    }
    static constexpr int total(int s) { return WARPS * (ring_bytes(s) + slot + 8 * s); }
    // stages (two records each) in flight per warp
    static constexpr int S = total(3) <= attn_smem(CTAS) ? 3 : 2;
    static constexpr int ring = ring_bytes(S);
    static constexpr int ring_off = 0;                     // [WARPS][ring]; later part 1 of a warp
    static constexpr int first_off = WARPS * ring;         // [WARPS][slot]: part 0
    static constexpr int bars_off = first_off + WARPS * slot;
    static constexpr int bytes = bars_off + WARPS * S * 8;
    static_assert(bytes <= attn_smem(CTAS), "the CTAs fit on an SM");
    static_assert(rec % 16 == 0 && slot % 16 == 0, "bulk copies and slots are 16-byte aligned");
    static_assert(2 * WARPS <= 32, "a lane per part");
};

struct Part {                          // a warp's part of an item
    int64_t item_begin, item_end;      // units; item_end = 0: none
    int cu0, n, h, rt;                 // the sequence's first query row and queries; head, row tile
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Larger of each half; a NaN is left out.
__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// c (+)= integer product of 4-bit codes (u8) with query bytes, m16n8k32.
template <bool ADD, bool SIGNED>
__device__ __forceinline__ void mma_i8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
    if (ADD) {
        if (SIGNED)
            asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 "
                "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
        else
            asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 "
                "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    } else {
        if (SIGNED)
            asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 "
                "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
        else
            asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.u8.s32 "
                "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
                : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(0));
    }
}
__device__ __forceinline__ float bf16_at(const uint8_t *q) {
    return __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t *>(q) << 16);
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(bar) : "memory");
}

// mbar_wait that reads the clock only after 64 polls (each may suspend the
// warp for up to a microsecond): the waits here are short and frequent.
__device__ __noinline__ bool ring_wait(uint32_t bar, uint32_t parity, uint64_t limit_ns,
                                       volatile uint32_t *abort_flag, unsigned int *err_word) {
    for (int i = 0; i < 64; ++i)
        if (mbar_try_wait_hint(bar, parity, 1000u)) return true;
    return mbar_wait(bar, parity, limit_ns, abort_flag, err_word);
}

// Output row of query row `row` of item (b, h), or null when there is none.
template <int D>
__device__ __forceinline__ uint16_t *out_row(const AttnArgs &p, int cu0, int n, int h, int row) {
    if (row >= n * p.share) return nullptr;
    const int i = row / p.share, tok = cu0 + i;
    if (tok < 0 || tok >= p.T) return nullptr;
    return p.out + (int64_t)tok * p.out_stride + (int64_t)(h * p.share + row - i * p.share) * D;
}

// Four results of a row (8-byte store where the row allows it).
__device__ __forceinline__ void store4(uint16_t *dst, float4 o, float f) {
    const uint32_t a = dev::pack_bf16x2(o.x * f, o.y * f), b = dev::pack_bf16x2(o.z * f, o.w * f);
    if ((reinterpret_cast<uintptr_t>(dst) & 7) == 0) {
        *reinterpret_cast<uint2 *>(dst) = make_uint2(a, b);
    } else {
        dst[0] = (uint16_t)a; dst[1] = (uint16_t)(a >> 16);
        dst[2] = (uint16_t)b; dst[3] = (uint16_t)(b >> 16);
    }
}

// Which groups of the lane's tokens (gid, gid + 8 of two records) hold zeros
// alone, as bits 4 group + 2 record + half.  Such a group has S = 1, Z = 0.
template <int D, int G>
__device__ __noinline__ uint32_t zero_groups(const uint8_t *r0, const uint8_t *r1, int lane) {
    constexpr int NG = D / G;
    const int gid = lane >> 2, tig = lane & 3;
    uint32_t zeros = 0u, ones = 0u;                // ones: S = 1
#pragma unroll
    for (int gr = 0; gr < NG; ++gr)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (*reinterpret_cast<const uint16_t *>((i >> 1 ? r1 : r0) + v_scales_off(D, NG) + 32 * gr +
                                                    2 * (gid + 8 * (i & 1))) == 0x3F80u)
                ones |= 1u << (4 * gr + i);
    const uint32_t some = __reduce_or_sync(0xFFFFFFFFu, ones);
#pragma unroll 1
    for (int gr = 0; gr < NG; ++gr) {
        if (!(some >> (4 * gr) & 15u)) continue;
        uint32_t bits[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint8_t *rec = i >> 1 ? r1 : r0;
            const int t = gid + 8 * (i & 1);
            bits[i] = rec[v_zeros_off(D, NG) + 16 * gr + t];
#pragma unroll
            for (int w = 0; w < (G < 64 ? 1 : G / 64); ++w)
#pragma unroll
                for (int u = 0; u < 4; ++u) {      // units 4 tig + u of a 64-wide span's 16
                    const uint32_t unit = *reinterpret_cast<const uint16_t *>(
                        rec + v_codes_off(D) +
                        v_unit_byte(D, t, gr * G / 64 + w, tig >> 1, 4 * (tig & 1) + u));
                    bits[i] |= G >= 64 ? unit : unit & (gr & 1 ? 0xFF00u : 0x00FFu);
                }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bits[i] |= __shfl_xor_sync(0xFFFFFFFFu, bits[i], 1);
            bits[i] |= __shfl_xor_sync(0xFFFFFFFFu, bits[i], 2);
            if (bits[i] == 0u) zeros |= 1u << (4 * gr + i);
        }
    }
    return zeros & ones;
}

// What a row's sums are multiplied with at the end: 1 / l; 0 for a row that
// saw no key, NaN when l is.
__device__ __forceinline__ float row_factor(float l) { return l > 0.0f ? 1.0f / l : l; }

template <int D, int G, int NB, int WARPS, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) kv4_attention_kernel(const AttnArgs p) {
    using L = AttnLayout<D, G, NB, WARPS, CTAS>;
    using SL = Slot<D, NB>;
    constexpr int NG = L::NG, S = L::S, R = 8 * NB, kThreads = 32 * WARPS;
    constexpr int KW = D / 32;                     // K words per token and lane; V words per lane and p
    constexpr int VW = D / 64;                     // 64-wide spans of d
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t pre[kThreads + 1];          // units before each thread's sequences
    __shared__ int64_t warp_sum[WARPS], warp_items[WARPS];
    __shared__ int warp_blocks[WARPS];
    __shared__ Part parts[2 * WARPS];
    __shared__ uint32_t abort_word;
    __shared__ int last_flag[2];
    volatile uint32_t *abort_flag = &abort_word;
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gid = lane >> 2, tig = lane & 3;
    auto work_of = [&](int b) {
        return seq_work(p.cu[b], p.cu[b + 1], p.kv_lens[b], p.T, p.capacity, p.window, p.share,
                        p.kv_heads, R);
    };

    // ---- units of all sequences: every CTA adds them up itself ----
    const int per = (p.B + kThreads - 1) / kThreads;           // sequences per thread
    int64_t scan = 0, items = 0;
    int blocks = 0;                                            // of the longest item
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b < p.B) {
            const SeqWork w = work_of(b);
            scan += w.units;
            items += w.row_tiles;
            if (w.n > 0) blocks = max(blocks, w.blocks);
            const int len = p.kv_lens[b];
            if (blockIdx.x == 0 && (len < 0 || len > p.capacity)) atomicOr(p.err_word, kErrIndex);
        }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
        if (lane >= o) scan += v;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) items += __shfl_xor_sync(0xFFFFFFFFu, items, o);
    blocks = __reduce_max_sync(0xFFFFFFFFu, blocks);
    if (lane == 31) {
        warp_sum[warp] = scan;
        warp_items[warp] = items;
        warp_blocks[warp] = blocks;
    }
    if (tid < 2 * WARPS) parts[tid].item_end = 0;
    if (tid == 0) abort_word = 0u;
    if (lane < S) mbar_init(sbase + L::bars_off + 8u * (warp * S + lane), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    int64_t before = 0, units = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += warp_sum[w];
        units += warp_sum[w];
        if (w != warp) {
            items += warp_items[w];
            blocks = max(blocks, warp_blocks[w]);
        }
    }
    pre[tid + 1] = before + scan;
    if (tid == 0) pre[0] = 0;
    __syncthreads();
    const int64_t quota =
        cta_quota(units, items * p.kv_heads, blocks, gridDim.x, p.min_units, p.whole_units);
    const int64_t cta_begin = range_begin(blockIdx.x, quota, units);
    const int64_t cta_end = range_begin(blockIdx.x + 1, quota, units);
    if (cta_begin >= cta_end) return;
    const int wq = warp_quota(cta_end - cta_begin, WARPS);
    const int64_t w_begin = min(cta_begin + (int64_t)warp * wq, cta_end);
    const int64_t w_end = min(w_begin + wq, cta_end);

    const uint32_t ring = sbase + L::ring_off + (uint32_t)warp * L::ring;
    const uint32_t bar0 = sbase + L::bars_off + 8u * (uint32_t)(warp * S);
    int stage = 0;                                 // next stage to consume
    uint32_t phase = 0;
    bool ok = true;
    int in_flight = 0;                             // stages to wait for after a failed wait

    if (w_begin < w_end) {
        // the sequence that holds unit w_begin: the last thread whose prefix is
        // not above it has units (threads without share the next one's prefix)
        int lo = 0;
        for (int i = lane; i < kThreads; i += 32)
            if (pre[i] <= w_begin) lo = i;
        lo = __reduce_max_sync(0xFFFFFFFFu, lo);
        int b = lo * per;
        int64_t seq_begin = pre[lo];
        SeqWork sw;
        for (;; ++b) {
            sw = work_of(b);
            if (w_begin < seq_begin + sw.units) break;
            seq_begin += sw.units;
        }
        int64_t u = w_begin;
        int item = (int)quotient(u - seq_begin, sw.blocks);         // (head, row tile) of the sequence
        while (u < w_end) {
            while (u >= seq_begin + sw.units) {                // next sequence with units
                seq_begin += sw.units;
                sw = work_of(++b);
                item = 0;
            }
            const int h = item / sw.row_tiles, rt = item - h * sw.row_tiles;
            const int64_t item_begin = seq_begin + (int64_t)item * sw.blocks;
            const int64_t item_end = item_begin + sw.blocks;
            const int64_t seg_end = min(item_end, w_end);
            const int blk0 = sw.block0 + (int)(u - item_begin);
            const int nblk = (int)(seg_end - u);
            const int steps = (nblk + 1) >> 1;                 // two blocks each
            const int cu0 = p.cu[b];
            const int32_t *table = p.page_table + (int64_t)b * p.max_pages;

            // ---- copies: step i's two records, lanes 0 and 1 one each ----
            // lane l holds the place of block 32 c + l of the segment, and of
            // block 32 (c + 1) + l
            const uint8_t *src_cur, *src_next;
            auto place = [&](int i) -> const uint8_t * {
                if (i >= nblk || (blk0 + i) * kBlock >= sw.len) return nullptr;
                const int64_t r = record_index(table, p.max_pages, p.num_pages, p.kv_heads, h,
                                               p.page_blocks, blk0 + i);
                return r < 0 ? nullptr : p.cache + r * L::rec;
            };
            src_next = place(lane);
            uint32_t have = 0;                     // two bits per stage: its records exist
            auto issue = [&](int i, int s) {       // step i into stage s
                if ((i & 15) == 0) {
                    src_cur = src_next;
                    src_next = place(2 * i + 32 + lane);
                }
                const uint8_t *src = reinterpret_cast<const uint8_t *>(__shfl_sync(
                    0xFFFFFFFFu, reinterpret_cast<unsigned long long>(src_cur), 2 * i + (lane & 1)));
                const uint32_t got = __ballot_sync(0xFFFFFFFFu, src != nullptr) & 3u;
                have = (have & ~(3u << (2 * s))) | got << (2 * s);
                if (lane < 2) {
                    const uint32_t bar = bar0 + 8u * s;
                    mbar_arrive_expect_tx(bar, src != nullptr ? (uint32_t)L::rec : 0u);
                    if (src != nullptr)
                        bulk_copy(ring + (uint32_t)(2 * s + lane) * L::rec, src, (uint32_t)L::rec, bar);
                }
            };
            // ---- queries: row gid of each 8-row tile ----
            uint4 qx[NB][KW];
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const int r = rt * R + 8 * nb + gid;
                const uint16_t *src = nullptr;
                if (r < sw.n * p.share) {
                    const int i = r / p.share, tok = cu0 + i;
                    if (tok < p.T)
                        src = p.q + (int64_t)tok * p.q_stride +
                              (int64_t)(h * p.share + r - i * p.share) * D + 8 * tig;
                }
#pragma unroll
                for (int j = 0; j < KW; ++j)
                    qx[nb][j] = src ? __ldg(reinterpret_cast<const uint4 *>(src + 32 * j))
                                    : make_uint4(0u, 0u, 0u, 0u);
            }
            for (int i = 0; i < S && i < steps; ++i) issue(i, stage + i < S ? stage + i : stage + i - S);

            // ---- queries as B fragments ----
            uint32_t qf[NB][4 * KW];
            float kq[NB][2];                       // per column 2 tig, 2 tig + 1
            int qsum[NG][NB][2];                   // sum_d i_d of each group
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
                const uint4 (&x)[KW] = qx[nb];
                uint32_t big = 0;                  // largest |q|, as bf16 bits (NaN above inf)
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        big = max(big, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
                }
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
                big = max(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
                // 2^e brings the largest |q| into [2^14, 2^15) (e <= 126)
                const int e = big ? min(14 + 127 - (int)(big >> 7), 126) : 0;
                const float f = __uint_as_float((uint32_t)(e + 127) << 23);
                int sum[NG];
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) sum[gr] = 0;
#pragma unroll
                for (int j = 0; j < KW; ++j) {
                    const uint32_t w[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                    int v[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[2 * i] = __float2int_rn(dev::bf16_lo(w[i]) * f);
                        v[2 * i + 1] = __float2int_rn(dev::bf16_hi(w[i]) * f);
                        sum[32 * j / G] += v[2 * i] + v[2 * i + 1];
                    }
                    // a word's even nibbles are k 4 tig .. of the product, its odd
                    // ones k 16 + 4 tig ..: high bytes, then low bytes
                    uint32_t f4[4];
#pragma unroll
                    for (int odd = 0; odd < 2; ++odd) {
                        const uint32_t a = dev::prmt(v[odd], v[2 + odd], 0x5140u);
                        const uint32_t c = dev::prmt(v[4 + odd], v[6 + odd], 0x5140u);
                        f4[odd] = dev::prmt(a, c, 0x7632u);        // high bytes
                        f4[2 + odd] = dev::prmt(a, c, 0x5410u);    // low bytes
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) qf[nb][4 * j + i] = f4[i];
                }
                // a row with an infinity or a NaN gives NaN
                const float kr = big >= 0x7F80u ? __int_as_float(0x7FFFFFFF)
                                                : p.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
                kq[nb][0] = __shfl_sync(0xFFFFFFFFu, kr, 8 * tig);
                kq[nb][1] = __shfl_sync(0xFFFFFFFFu, kr, 8 * tig + 4);
#pragma unroll
                for (int gr = 0; gr < NG; ++gr) {
                    int t = sum[gr];
                    t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
                    t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
                    qsum[gr][nb][0] = __shfl_sync(0xFFFFFFFFu, t, 8 * tig);
                    qsum[gr][nb][1] = __shfl_sync(0xFFFFFFFFu, t, 8 * tig + 4);
                }
            }
            // keys that all rows, and that any row, of the tile may see
            const int pos0 = first_position(p.kv_lens[b], sw.n);
            const int r0 = rt * R, r1 = min(r0 + R, sw.n * p.share) - 1;
            const int all_hi = pos0 + r0 / p.share + 1, any_hi = pos0 + r1 / p.share + 1;
            const int all_lo = p.window > 0 ? max(any_hi, 0) - p.window : 0;

            // ---- main loop ----
            float acc[4 * VW][NB][4], l[NB][2], m[NB][2];
            float vf[NG][NB][2];                   // 2^-E
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
                for (int i = 0; i < 4 * VW; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[i][nb][c] = 0.0f;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    l[nb][c] = 0.0f;
                    m[nb][c] = kNoMax;
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) vf[gr][nb][c] = 0x1p126f;
                }
            }
            for (int i = 0; i < steps; ++i) {
                if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(bar0 + 8u * stage, phase))) {
                    ok = ring_wait(bar0 + 8u * stage, phase, p.wait_limit, abort_flag, p.err_word);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) {
                        in_flight = min(S, steps - i);
                        break;
                    }
                }
                const int key0 = (blk0 + 2 * i) * kBlock;
                const uint32_t got = (have >> (2 * stage)) & 3u;
                if (key0 < any_hi && got != 0) {
                    // a record that was not copied holds an earlier one's bytes
                    // (or none yet): all its keys are masked
                    const uint8_t *st0 = smem + L::ring_off + warp * L::ring + 2 * stage * L::rec;
                    const uint8_t *sr[2] = {got == 2u ? st0 + L::rec : st0,
                                            got == 1u ? st0 : st0 + L::rec};
                    float s[2][NB][4], vs[2][NG][2];
                    // -- scores (without kq): tokens gid and gid + 8 of each
                    //    record, columns 2 tig, 2 tig + 1
                    uint32_t kw[2][2][KW];
#pragma unroll
                    for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                        for (int q = 0; q < (2 * KW + 3) / 4; ++q) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                sr[rc] + k_codes_off() + q * 512 + lane * 16);
                            const uint32_t t[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                kw[rc][(4 * q + x) / KW][(4 * q + x) % KW] = t[x];
                        }
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr) {
                        int th[2][NB][4], tl[2][NB][4];    // high and low bytes of the queries
#pragma unroll
                        for (int jj = 0; jj < G / 32; ++jj) {
                            const int j = gr * (G / 32) + jj;
#pragma unroll
                            for (int rc = 0; rc < 2; ++rc) {
                                const uint32_t a = kw[rc][0][j], c = kw[rc][1][j];
                                const uint32_t a0 = a & 0x0F0F0F0Fu, a1 = c & 0x0F0F0F0Fu;
                                const uint32_t a2 = (a >> 4) & 0x0F0F0F0Fu, a3 = (c >> 4) & 0x0F0F0F0Fu;
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    if (jj == 0) {
                                        mma_i8<false, true>(th[rc][nb], a0, a1, a2, a3, qf[nb][4 * j], qf[nb][4 * j + 1]);
                                        mma_i8<false, false>(tl[rc][nb], a0, a1, a2, a3, qf[nb][4 * j + 2], qf[nb][4 * j + 3]);
                                    } else {
                                        mma_i8<true, true>(th[rc][nb], a0, a1, a2, a3, qf[nb][4 * j], qf[nb][4 * j + 1]);
                                        mma_i8<true, false>(tl[rc][nb], a0, a1, a2, a3, qf[nb][4 * j + 2], qf[nb][4 * j + 3]);
                                    }
                                }
                            }
                        }
#pragma unroll
                        for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int z = sr[rc][k_zeros_off(D, NG) + 16 * gr + gid + 8 * x];
                                const float sc = bf16_at(sr[rc] + k_scales_off(D) + 32 * gr + 2 * (gid + 8 * x));
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                    for (int c = 0; c < 2; ++c) {
                                        const float t = (float)(th[rc][nb][2 * x + c] * 256 +
                                                                tl[rc][nb][2 * x + c] -
                                                                z * qsum[gr][nb][c]);
                                        s[rc][nb][2 * x + c] =
                                            gr == 0 ? t * sc : fmaf(t, sc, s[rc][nb][2 * x + c]);
                                    }
                            }
                    }
                    // -- V scales
#pragma unroll
                    for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int gr = 0; gr < NG; ++gr)
                                vs[rc][gr][x] =
                                    bf16_at(sr[rc] + v_scales_off(D, NG) + 32 * gr + 2 * (gid + 8 * x));
                    // -- scores in powers of two, masks
#pragma unroll
                    for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[rc][nb][c] *= kq[nb][c & 1];
                    if (got != 3u || key0 < all_lo || key0 + 2 * kBlock > all_hi) {
                        if (lane == 0)
                            for (int rc = 0; rc < 2; ++rc)      // existing keys without a page
                                if (!((got >> rc) & 1u) && 2 * i + rc < nblk && key0 + 16 * rc < sw.len)
                                    atomicOr(p.err_word, kErrIndex);
                        bool wild = false;
                        // keys each column's row may see: [klo, khi)
                        int khi[NB][2], klo[NB][2];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                khi[nb][c] = pos0 + min(r0 + 8 * nb + 2 * tig + c, r1) / p.share + 1;
                                klo[nb][c] = p.window > 0 ? max(khi[nb][c], 0) - p.window : 0;
                            }
#pragma unroll
                        for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const int key = key0 + 16 * rc + gid + 8 * x;
                                const bool none = !((got >> rc) & 1u) || key >= sw.len;
                                if (none) {                     // not written, whatever it holds
#pragma unroll
                                    for (int gr = 0; gr < NG; ++gr) vs[rc][gr][x] = 0.0f;
                                }
#pragma unroll
                                for (int gr = 0; gr < NG; ++gr) wild |= !(vs[rc][gr][x] <= 3.4e38f);
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
                                        if (none || key >= khi[nb][c] || key < klo[nb][c])
                                            s[rc][nb][2 * x + c] = __int_as_float(0xFF800000);
                            }
                        // a scale that is not finite (values that were not) makes its group
                        // NaN in the rows that see the key, as it does in a step that all see,
                        // and may not reach the others through 0 * inf
                        if (__any_sync(0xFFFFFFFFu, wild)) {
                            uint32_t spoilt = 0u;              // groups of columns
#pragma unroll
                            for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
#pragma unroll
                                    for (int gr = 0; gr < NG; ++gr)
                                        if (!(vs[rc][gr][x] <= 3.4e38f)) {
                                            vs[rc][gr][x] = 0.0f;
#pragma unroll
                                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                                for (int c = 0; c < 2; ++c)
                                                    if (s[rc][nb][2 * x + c] != __int_as_float(0xFF800000))
                                                        spoilt |= 1u << (NG * (2 * nb + c) + gr);
                                        }
#pragma unroll
                            for (int o = 4; o < 32; o <<= 1) spoilt |= __shfl_xor_sync(0xFFFFFFFFu, spoilt, o);
#pragma unroll
                            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
#pragma unroll
                                    for (int z = 0; z < 4 * VW; ++z)
                                        if (spoilt >> (NG * (2 * nb + c) + 16 * z / G) & 1u)
                                            acc[z][nb][c] = acc[z][nb][c + 2] = __int_as_float(0x7FFFFFFF);
                        }
                    }
                    // -- weights 2^(s - m) S 2^-E in fp16, pairs of columns: s is kept
                    //    for the case that m moves
                    uint32_t w[2][NG][NB][2];
                    float lt[NB][2];
                    bool raise;
                    auto weights = [&]() {
                        uint32_t top = 0u;                      // pair of the largest (NaN left out)
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb) lt[nb][0] = lt[nb][1] = 0.0f;
#pragma unroll
                        for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
#pragma unroll
                                for (int nb = 0; nb < NB; ++nb) {
                                    const float q0 = ex2(s[rc][nb][2 * x] - m[nb][0]);
                                    const float q1 = ex2(s[rc][nb][2 * x + 1] - m[nb][1]);
                                    lt[nb][0] += q0;
                                    lt[nb][1] += q1;
#pragma unroll
                                    for (int gr = 0; gr < NG; ++gr) {
                                        const float S = vs[rc][gr][x];   // first: 0 keeps q 2^-E finite
                                        w[rc][gr][nb][x] = pack_f16x2(q0 * S * vf[gr][nb][0],
                                                                      q1 * S * vf[gr][nb][1]);
                                        top = max_f16x2(top, w[rc][gr][nb][x]);
                                    }
                                }
                        // 2^12 as fp16; l stays far from fp32's end
                        raise = (top & 0xFFFFu) >= 0x6C00u || top >= 0x6C000000u;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
                            raise |= fmaxf(lt[nb][0], lt[nb][1]) >= 0x1p100f;
                    };
                    // a second pass when groups of zeros have left, a last one when m and
                    // E have moved
                    bool moved = false, cleared = false;
#pragma unroll 1
                    for (;;) {
                        weights();
                        if (!__any_sync(0xFFFFFFFFu, raise) || moved) break;
                        if (!cleared) {
                            cleared = true;
                            // a group of zeros is stored with S = 1, Z = 0 and adds nothing:
                            // it sets no E
                            bool one = false;
#pragma unroll
                            for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
#pragma unroll
                                    for (int gr = 0; gr < NG; ++gr) one |= vs[rc][gr][x] == 1.0f;
                            if (__any_sync(0xFFFFFFFFu, one)) {
                                const uint32_t zeros = zero_groups<D, G>(sr[0], sr[1], lane);
#pragma unroll
                                for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                                    for (int x = 0; x < 2; ++x)
#pragma unroll
                                        for (int gr = 0; gr < NG; ++gr)
                                            if (zeros >> (4 * gr + 2 * rc + x) & 1u) vs[rc][gr][x] = 0.0f;
                                continue;
                            }
                        }
                        moved = true;
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float d = fmaxf(fmaxf(s[0][nb][c], s[0][nb][c + 2]),
                                                fmaxf(s[1][nb][c], s[1][nb][c + 2]));
#pragma unroll
                                for (int o = 4; o < 32; o <<= 1)
                                    d = fmaxf(d, __shfl_xor_sync(0xFFFFFFFFu, d, o));
                                d = fmaxf(d, m[nb][c]);
                                const float down = m[nb][c] - d;
                                m[nb][c] = d;
                                l[nb][c] *= ex2(down);
#pragma unroll
                                for (int gr = 0; gr < NG; ++gr) {
                                    float top = 0.0f;           // the largest weight
#pragma unroll
                                    for (int rc = 0; rc < 2; ++rc)
#pragma unroll
                                        for (int x = 0; x < 2; ++x)
                                            top = fmaxf(top, ex2(s[rc][nb][2 * x + c] - d) * vs[rc][gr][x]);
#pragma unroll
                                    for (int o = 4; o < 32; o <<= 1)
                                        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                                    // E follows the weights so far down when m moves: a key
                                    // that no longer counts does not set the rounding
                                    const int old = 127 - (int)(__float_as_uint(vf[gr][nb][c]) >> 23);
                                    int e = (int)(__float_as_uint(top) >> 23) - 127;
                                    e = max(e, old + (int)floorf(fmaxf(down, -300.0f)));
                                    e = min(max(e, -126), 100);
                                    const float f = ex2(down + (float)(old - e));
#pragma unroll
                                    for (int z = gr * G / 16; z < (gr + 1) * G / 16; ++z) {
                                        acc[z][nb][c] *= f;
                                        acc[z][nb][c + 2] *= f;
                                    }
                                    vf[gr][nb][c] = __uint_as_float((uint32_t)(127 - e) << 23);
                                }
                            }
                    }
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb) {
                        l[nb][0] += lt[nb][0];
                        l[nb][1] += lt[nb][1];
                    }
                    // -- values: rows d, columns 2 tig, 2 tig + 1
#pragma unroll
                    for (int rc = 0; rc < 2; ++rc) {
                        const uint8_t *st = sr[rc];
                        uint32_t wf[NG][NB][2];
#pragma unroll
                        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                            for (int x = 0; x < 2; ++x)
#pragma unroll
                                for (int gr = 0; gr < NG; ++gr)
                                    wf[gr][nb][x] = transpose8(w[rc][gr][nb][x]);
                        uint32_t vw[2][KW];
#pragma unroll
                        for (int q = 0; q < (2 * KW + 3) / 4; ++q) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                st + v_codes_off(D) + q * 512 + lane * 16);
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
                                    *reinterpret_cast<const uint16_t *>(st + v_zeros_off(D, NG) + 16 * gr + 8 * x + 2 * tig),
                                    0u, 0x4140u);
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
                } else if (key0 < any_hi && lane == 0 && key0 < sw.len) {
                    atomicOr(p.err_word, kErrIndex);           // neither record has a page
                }
                // every register loaded from the stage has been consumed by an
                // MMA or a conversion: it may be filled again
                __syncwarp();
                if (i + S < steps) issue(i + S, stage);
                if (++stage == S) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;

            // ---- the segment's result: rows of sums, in this warp's idle ring, or
            // beside it when the item began in front of this warp's range and
            // ends inside it (the ring goes on to serve)
            const bool whole = u == item_begin && seg_end == item_end;
            const int which = whole || seg_end == w_end ? 1 : 0;
            float *slot = reinterpret_cast<float *>(
                smem + (which ? L::ring_off + warp * L::ring : L::first_off + warp * L::slot));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = 8 * nb + 2 * tig + c;
                    float t = l[nb][c];
                    float back[NG];                          // 2^E
#pragma unroll
                    for (int gr = 0; gr < NG; ++gr)
                        back[gr] = __uint_as_float((254u << 23) - __float_as_uint(vf[gr][nb][c]));
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
                    if (gid == 0) {
                        slot[SL::stats + row] = m[nb][c];
                        slot[SL::stats + R + row] = t;
                    }
#pragma unroll
                    for (int wi = 0; wi < VW; ++wi)
#pragma unroll
                        for (int nib = 0; nib < 4; ++nib)
#pragma unroll
                            for (int hi = 0; hi < 2; ++hi)
                                slot[row * SL::pitch + 64 * wi + 16 * nib + 8 * hi + gid] =
                                    acc[4 * wi + nib][nb][2 * hi + c] * back[(64 * wi + 16 * nib) / G];
                }
            if (whole) {
                __syncwarp();
                for (int e = lane; e < R * D / 4; e += 32) {
                    const int row = e / (D / 4), d = 4 * (e % (D / 4));
                    if (uint16_t *dst = out_row<D>(p, cu0, sw.n, h, rt * R + row))
                        store4(dst + d, *reinterpret_cast<const float4 *>(slot + row * SL::pitch + d),
                               row_factor(slot[SL::stats + R + row]));
                }
                // the ring's next copies come behind these accesses
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
            } else if (lane == 0) {
                parts[2 * warp + which] = Part{item_begin, item_end, cu0, sw.n, h, rt};
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
    // lane i < 2 WARPS stands for parts[i]; `heads`: the first part of each item
    const int64_t my_end = lane < 2 * WARPS ? parts[lane].item_end : 0;
    const int64_t my_begin = lane < 2 * WARPS ? parts[lane].item_begin : 0;
    const uint32_t valid = __ballot_sync(0xFFFFFFFFu, my_end != 0);
    const uint32_t below = valid & ((1u << lane) - 1u);
    const int64_t prev_begin = __shfl_sync(0xFFFFFFFFu, my_begin, below ? 31 - __clz(below) : 0);
    const uint32_t heads = __ballot_sync(0xFFFFFFFFu, my_end != 0 && (!below || prev_begin != my_begin));
    const uint32_t shared = __ballot_sync(
        0xFFFFFFFFu, my_end != 0 && (my_begin < cta_begin || my_end > cta_end));
    auto slot_of = [&](int i) {                     // of parts[i]
        return reinterpret_cast<const float *>(
            smem + ((i & 1) ? L::ring_off + (i >> 1) * L::ring : L::first_off + (i >> 1) * L::slot));
    };
    // CG threads per row, each 16-byte pieces of it; groups of threads that
    // cover all rows take items in turn
    constexpr int CG = D / 4 < kThreads / R ? D / 4 : kThreads / R, kGroups = kThreads / (R * CG);
    constexpr int DI = (D / 4 + CG - 1) / CG;       // pieces per thread
    const int grp = tid / (R * CG), row = tid % (R * CG) / CG, piece0 = tid % CG;
    int turn = 0;
    for (uint32_t todo = heads; todo; todo &= todo - 1, ++turn) {
        if (grp != turn % kGroups) continue;
        const int i = __ffs(todo) - 1;
        const uint32_t rest = todo & (todo - 1);
        const uint32_t mine = valid & (rest ? (1u << (__ffs(rest) - 1)) - 1u : ~0u) & ~((1u << i) - 1u);
        const Part &it = parts[i];
        if (it.rt * R + row >= it.n * p.share) continue;
        float mx = kNoMax, l = 0.0f;
        float4 o[DI];
#pragma unroll
        for (int y = 0; y < DI; ++y) o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (uint32_t x = mine; x; x &= x - 1) mx = fmaxf(mx, slot_of(__ffs(x) - 1)[SL::stats + row]);
        for (uint32_t x = mine; x; x &= x - 1) {
            const float *q = slot_of(__ffs(x) - 1);
            const float w = ex2(q[SL::stats + row] - mx);
            l += w * q[SL::stats + R + row];
#pragma unroll
            for (int y = 0; y < DI; ++y) {
                const int d = 4 * (piece0 + y * CG);
                if (DI * CG > D / 4 && d >= D) break;
                const float4 v = *reinterpret_cast<const float4 *>(q + row * SL::pitch + d);
                o[y].x += w * v.x; o[y].y += w * v.y; o[y].z += w * v.z; o[y].w += w * v.w;
            }
        }
        const bool out_of_cta = (shared >> i) & 1u;
        float *part_dst = p.partials + ((int64_t)blockIdx.x * 2 +
                                        partial_slot(it.item_begin, cta_begin)) * SL::floats;
        uint16_t *dst = out_row<D>(p, it.cu0, it.n, it.h, it.rt * R + row);
        if (out_of_cta && piece0 == 0) {
            __stcg(part_dst + SL::stats + row, mx);
            __stcg(part_dst + SL::stats + R + row, l);
        }
#pragma unroll
        for (int y = 0; y < DI; ++y) {
            const int d = 4 * (piece0 + y * CG);
            if (DI * CG > D / 4 && d >= D) break;
            if (out_of_cta)
                __stcg(reinterpret_cast<float4 *>(part_dst + row * SL::pitch + d), o[y]);
            else if (dst)
                store4(dst + d, o[y], row_factor(l));
        }
    }
    if (!shared) return;
    // ---- items shared by CTAs: the last to arrive adds the parts in order ----
    const uint32_t ends = heads & shared;           // one or two items
    __syncthreads();
    if (tid < 2) {
        last_flag[tid] = 0;
        const uint32_t x = tid ? ends & (ends - 1) : ends;
        if (x) {
            const Part &it = parts[__ffs(x) - 1];
            const int64_t c0 = quotient(it.item_begin, quota);
            const int64_t c1 = quotient(it.item_end - 1, quota);
            __threadfence();                        // this CTA's parts, ordered by the barrier
            last_flag[tid] = atomicAdd(&p.counters[c0], 1u) == (uint32_t)(c1 - c0);
            __threadfence();
        }
    }
    __syncthreads();
    for (int k = 0; k < 2; ++k) {
        if (!last_flag[k]) continue;
        const Part it = parts[__ffs(k ? ends & (ends - 1) : ends) - 1];
        const int64_t c0 = quotient(it.item_begin, quota);
        const int count = (int)(quotient(it.item_end - 1, quota) - c0) + 1;
        const int s0 = partial_slot(it.item_begin, range_begin(c0, quota, units));
        const float *base = p.partials + 2 * c0 * SL::floats;
        auto part = [&](int x) { return base + (int64_t)(2 * x + (x == 0 ? s0 : 0)) * SL::floats; };
        uint16_t *dst = out_row<D>(p, it.cu0, it.n, it.h, it.rt * R + row);
        if (grp == k % kGroups && dst) {
            float mx = kNoMax, l = 0.0f;
            float4 o[DI];
#pragma unroll
            for (int y = 0; y < DI; ++y) o[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            // U parts at a time, their loads together
            constexpr int U = DI == 1 ? 10 : DI <= 4 ? 4 : 2;
            for (int x0 = 0; x0 < count; x0 += U) {
                float pm[U], pl[U];
                float4 v[U][DI];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float *q = part(min(x0 + u, count - 1));
                    pm[u] = __ldcg(q + SL::stats + row);
                    pl[u] = __ldcg(q + SL::stats + R + row);
#pragma unroll
                    for (int y = 0; y < DI; ++y) {
                        const int d = 4 * min(piece0 + y * CG, D / 4 - 1);
                        v[u][y] = __ldcg(reinterpret_cast<const float4 *>(q + row * SL::pitch + d));
                    }
                }
                float m2 = mx;
#pragma unroll
                for (int u = 0; u < U; ++u) m2 = fmaxf(m2, pm[u]);
                const float f = ex2(mx - m2);
                mx = m2;
                l *= f;
#pragma unroll
                for (int y = 0; y < DI; ++y) { o[y].x *= f; o[y].y *= f; o[y].z *= f; o[y].w *= f; }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float w = x0 + u < count ? ex2(pm[u] - mx) : 0.0f;
                    l += w * pl[u];
#pragma unroll
                    for (int y = 0; y < DI; ++y) {
                        o[y].x += w * v[u][y].x; o[y].y += w * v[u][y].y;
                        o[y].z += w * v[u][y].z; o[y].w += w * v[u][y].w;
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < DI; ++y) {
                const int d = 4 * (piece0 + y * CG);
                if (DI * CG > D / 4 && d >= D) break;
                store4(dst + d, o[y], row_factor(l));
            }
        }
        if (tid == 0) p.counters[c0] = 0u;
    }
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
// CTAs per SM, and warps per CTA so that the accumulators, the queries and what
// each group of channels needs stay in registers, but for a few words.
// D = 128, warm: one CTA of 12 warps against two of 6, half the parts to join:
// one sequence of 131001 tokens 49, 59 us, 128 sequences 165, 173.  D = 64 has many
// short items and takes two: 17 sequences of draft tokens 28.5 us, with one CTA of 16
// warps 29.8.  64 x 4000 tokens, 8 key heads of 128, 4 query heads each, warm: groups
// of 32 94 us with 12 warps, 121 with 14 of 128 registers; of 64 76, 81 with 16; of
// 128 68, 71 with 16.  16-row tiles of groups of 32 (16 query heads): 137 with 4
// warps, 190 with 6.
constexpr int kAttnCtasPerSm = 2;      // at most
template <int D, int NB>
constexpr int kAttnCtas = D == 128 && NB == 1 ? 1 : kAttnCtasPerSm;
template <int D, int G, int NB>
constexpr int kAttnWarps =
    D == 256 ? 4 : NB == 2 ? (D == 128 ? 4 : 6) : D == 64 ? 8 : 12;

// Rows of a tile: 8 or 16.  A tile of 16 reads and unpacks the keys once for
// twice the rows, but has half the warps per CTA and twice the products and
// softmax per step.  Warm, 8 key heads, 8- against 16-row tiles, us:
//                     64 x 4000 tokens,       1 x 32000 tokens,
//                     16 rows   512 rows      16 rows   128 rows  per key head
//   D = 64,  g = 32   104  87   2667  2096    27  35     99   85
//   D = 64,  g = 64    88  71   2293  1695    24  33     85   70
//   D = 128, g = 32   166 137   4701  3593    38  48    163  134
//   D = 128, g = 64   132 109   3949  2816    35  43    133  107
//   D = 128, g = 128  119  98   3538  2530    32  40    118   97
//   D = 256, g = 64   241 366   7941 10746     -         227  356
//   D = 256, g = 128  199 277   6855  7967     -         238  269
// 16 when a sequence has more than 8 rows on average and the 8-row tiles come to
// 128 or more (below that the longer tiles leave the machine idle), for 64-wide
// heads and for groups of 32.  The rule is older than the four warps of 128-wide
// tiles, with which groups of 64 and 128 would gain as well.
template <int D, int G>
constexpr bool kTallTiles = D == 64 || G == 32;
bool tall_tiles(const AttnArgs &p) {
    const int64_t rows = (int64_t)p.T * p.share;
    return rows > 8 * (int64_t)p.B && rows * p.kv_heads >= 8 * 128;
}

template <int D, int G, int NB>
qz_status launch_attn(const AttnArgs &in, cudaStream_t st) {
    constexpr int W = kAttnWarps<D, G, NB>, C = kAttnCtas<D, NB>;
    using L = AttnLayout<D, G, NB, W, C>;
    auto kernel = kv4_attention_kernel<D, G, NB, W, C>;
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
    // two steps of two blocks per warp at least, as a CTA's prologue and join
    // outweigh a shorter loop.  Eight sequences of 100..3000 tokens, 32 query and 8 key
    // heads of 128, warm: 2, 4, 8 units per warp 20.6, 20.6, 21.4 us; one of 32000 or
    // 131001, 64 of 4000, drafts with a window and a mixed batch alike.
    AttnArgs args = in;
    args.min_units = 4 * W;
    // items alike of up to six steps per warp whole in a CTA, not cut: one
    // sequence of 777 tokens 10.8 us, cut 17.5; the calls above alike
    args.whole_units = 12 * W;
    kernel<<<(unsigned)(device_sm_count() * C), 32 * W, L::bytes, st>>>(args);
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

// One wave of CTAs, and no more than there can be warps with work (a call's
// tokens lie in at most T / 16 + 2 B blocks).
template <typename K>
qz_status launch_store(K kernel, int per_warp, int ctas_per_sm, const StoreArgs &p,
                       DeviceOnce &once, cudaStream_t st) {
    const int smem = per_warp * kStoreWarps;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return QZ_ERR_CUDA;
    }
    if (once.run(dev, [&] {
            cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
            return e;
        }) != cudaSuccess)
        return QZ_ERR_CUDA;
    const int64_t most = ceil_div(((int64_t)p.T / kBlock + 2 * (int64_t)p.B) * p.kv_heads, kStoreWarps);
    const int64_t fit = (int64_t)device_sm_count() * ctas_per_sm;
    kernel<<<(unsigned)(most < fit ? most : fit), kStoreThreads, smem, st>>>(p);
    return launch_status();
}
template <int D, int G>
struct Append {
    static qz_status go(const StoreArgs &p, cudaStream_t st) {
        static DeviceOnce once;
        return launch_store(kv4_append_kernel<D, G>, StoreLayout<D, G>::per_warp, kAppendCtas, p, once, st);
    }
};
template <int D, int G>
struct Read {
    static qz_status go(const StoreArgs &p, cudaStream_t st) {
        static DeviceOnce once;
        return launch_store(kv4_read_kernel<D, G>, StoreLayout<D, G>::per_warp, kReadCtas<D>, p, once, st);
    }
};
template <int D, int G>
struct Attend {
    static qz_status go(const AttnArgs &p, cudaStream_t st) {
        if constexpr (kTallTiles<D, G>)
            if (tall_tiles(p)) return launch_attn<D, G, 2>(p, st);
        return launch_attn<D, G, 1>(p, st);
    }
};

StoreArgs store_args(const Kv4Cache &c) {
    StoreArgs p{};
    p.cache = static_cast<uint8_t *>(c.cache);
    p.page_table = static_cast<const int32_t *>(c.page_table);
    p.kv_lens = static_cast<const int32_t *>(c.kv_lens);
    p.cu = static_cast<const int32_t *>(c.cu);
    p.T = (int)c.T; p.B = (int)c.B;
    p.max_pages = c.max_pages; p.num_pages = c.num_pages;
    p.kv_heads = (int)c.kv_heads; p.page_blocks = (int)(c.page_size / kBlock);
    p.err_word = device_error_word();
    return p;
}

size_t slot_bytes(int64_t D, int tiles) { return (size_t)(8 * tiles * (D + 4) + 16 * tiles) * 4; }

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
    return dispatch<Append>(c.head_dim, c.group_size, p, st);
}

qz_status launch_kv4_read(const Kv4Cache &c, void *k, void *v, cudaStream_t st) {
    StoreArgs p = store_args(c);
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    p.k_out = static_cast<uint16_t *>(k);
    p.v_out = static_cast<uint16_t *>(v);
    return dispatch<Read>(c.head_dim, c.group_size, p, st);
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
    p.T = (int)c.T; p.B = (int)c.B;
    p.max_pages = c.max_pages; p.num_pages = c.num_pages;
    constexpr int64_t kMaxLen = (int64_t(1) << 31) - 128;   // positions of a step stay below 2^31
    p.capacity = (int)(c.max_pages * c.page_size < kMaxLen ? c.max_pages * c.page_size : kMaxLen);
    p.window = window < p.capacity ? (int)window : 0;      // reaches every key: none
    p.kv_heads = (int)c.kv_heads;
    p.share = (int)(q_heads / c.kv_heads);
    p.page_blocks = (int)(c.page_size / kBlock);
    p.scale_log2 = (float)((double)scale * 1.4426950408889634);
    p.out = static_cast<uint16_t *>(out);
    p.out_stride = out_stride;
    // counters first: their place does not depend on the tile size
    p.counters = static_cast<uint32_t *>(workspace);
    p.partials = reinterpret_cast<float *>(static_cast<char *>(workspace) + kCounterBytes);
    p.wait_limit = device_wait_limit();
    p.err_word = device_error_word();
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    return dispatch<Attend>(c.head_dim, c.group_size, p, st);
}

}  // namespace qz
