// qz_lora.cu -- low-rank adapters of many requests beside a packed projection:
//   y_m = bf16( sum_k a_mk w^_nk + s_r sum_j B_r[n][j] h_mj ),  h_mj = sum_k A_r[j][k] a_mk,
// r the adapter of token m.  This kernel makes h; the GEMV adds the second
// product to its sums (qz_gemv.cu, LORA), so the output is rounded once.
//
// Tokens that share an adapter are worked on together, so each adapter in use
// is read once: every warp finds the adapters and their tokens from the M
// indices itself (qz_lora.cuh).  The product runs on mma.sync m16n8k16 with
// bf16 operands and fp32 sums: 16 ranks x 8 tokens, up
// to 16 tokens at a time.  The fragments' k order is
// free as long as both operands agree, so a lane reads 16 consecutive bytes of
// a row: k = 8 tid .. 8 tid + 7 of every 32.  A cluster of 8 blocks takes 16
// ranks of one adapter; the blocks and their 8 warps share K, and their sums
// meet in shared memory, the cluster's in its first block, in a fixed order.
// h (times s_r) is kept as two bf16 values, h = hi + lo (2^-17 of h), the
// operands of the second product.
//
// Bound by latency.  Alone, warm: 11 adapters of rank 64, K = 8192 (11.5 MB of
// A) 8.9 us; 9 of rank 32, K = 4096 6.2 us; one of rank 16 4.1 us.  The GEMV is
// launched beside it and waits only before it uses h.
#include <cuda_runtime.h>

#include "qz_lora.cuh"
#include "qz_lora_index.cuh"
#include "qz_serving.cuh"

namespace qz {
namespace {

constexpr unsigned kErrIndex = 2u;     // bit of the device error word: adapter index out of range
constexpr int kDownWarps = 8;
constexpr int kCluster = 8;
static_assert(32 * kDownWarps == 16 * 16, "a thread per rank and token");

struct LoraArgs {
    const uint16_t *a, *down;          // M x K; adapters x R x K
    const int32_t *ids;
    const float *scales;
    int M, K, R, adapters;
    uint16_t *h;                       // [2][M][R]: hi, lo
    unsigned int *err_word;
};

__device__ __forceinline__ void grid_release() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The c-th lowest token of the mask, -1 when there are fewer.
__device__ __forceinline__ int nth_token(uint64_t mask, int c) {
    for (int i = 0; i < c; ++i) mask &= mask - 1;
    return mask ? __ffsll((long long)mask) - 1 : -1;
}

__device__ __forceinline__ uint64_t drop_tokens(uint64_t mask, int n) {
    for (int i = 0; i < n && mask; ++i) mask &= mask - 1;
    return mask;
}

// Value at the same place of shared memory in block `rank` of the cluster.
__device__ __forceinline__ float cluster_load(const float *p, uint32_t rank) {
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p));
    float v;
    asm volatile("{\n\t.reg .u32 r;\n\tmapa.shared::cluster.u32 r, %1, %2;\n\t"
                 "ld.shared::cluster.f32 %0, [r];\n\t}" : "=f"(v) : "r"(a), "r"(rank) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---------------------------------------------------------------------------
// down: grid (adapters in use at most, ceil(R / 16), 8), clusters along z
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(32 * kDownWarps) __cluster_dims__(1, 1, kCluster)
lora_down_kernel(const LoraArgs p) {
    grid_release();
    __shared__ float part[kDownWarps][16 * 16], sums[16 * 16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
    const int j0 = 16 * blockIdx.y, rank = blockIdx.z;
    if (blockIdx.x == 0 && j0 == 0 && rank == 0 && threadIdx.x < p.M &&
        p.ids[threadIdx.x] >= p.adapters)
        atomicOr(p.err_word, kErrIndex);
    lora::Groups it(p.ids, p.M, p.adapters, lane);
    it.skip(blockIdx.x);
    if (!it.next()) return;                                  // the whole cluster
    const int id = it.id;
    uint64_t mask = it.tokens;
    const float scale = p.scales[id];
    const uint16_t *row0 = p.down + ((int64_t)id * p.R + j0 + gid) * p.K + 8 * tid;
    const uint16_t *row1 = row0 + (int64_t)8 * p.K;
    const bool v0 = j0 + gid < p.R, v1 = j0 + gid + 8 < p.R;
    const int steps = p.K / 32;                              // K is a multiple of 128
    const int w = rank * kDownWarps + warp;
    const int s0 = lora::part_begin(w, steps, kCluster * kDownWarps);
    const int s1 = lora::part_begin(w + 1, steps, kCluster * kDownWarps);
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    while (mask) {
        const bool two = __popcll(mask) > 8;
        const int tok0 = nth_token(mask, gid), tok1 = nth_token(mask, gid + 8);   // columns gid, gid + 8
        const uint16_t *act0 = p.a + (int64_t)max(tok0, 0) * p.K + 8 * tid;
        const uint16_t *act1 = p.a + (int64_t)max(tok1, 0) * p.K + 8 * tid;
        float acc[2][4] = {};
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const uint4 x = v0 ? dev::ld_stream_v4(row0 + 32 * s) : none;
            const uint4 y = v1 ? dev::ld_stream_v4(row1 + 32 * s) : none;
            const uint4 b = tok0 >= 0 ? __ldg(reinterpret_cast<const uint4 *>(act0 + 32 * s)) : none;
            dev::mma_bf16_16816(acc[0], x.x, y.x, x.y, y.y, b.x, b.y);
            dev::mma_bf16_16816(acc[0], x.z, y.z, x.w, y.w, b.z, b.w);
            if (two) {
                const uint4 c = tok1 >= 0 ? __ldg(reinterpret_cast<const uint4 *>(act1 + 32 * s)) : none;
                dev::mma_bf16_16816(acc[1], x.x, y.x, x.y, y.y, c.x, c.y);
                dev::mma_bf16_16816(acc[1], x.z, y.z, x.w, y.w, c.z, c.w);
            }
        }
        // acc[c][i]: rank gid + 8 (i >> 1), token column 8 c + 2 tid + (i & 1)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                part[warp][(gid + 8 * (i >> 1)) * 16 + 8 * c + 2 * tid + (i & 1)] = acc[c][i];
        __syncthreads();
        {
            float h = 0.0f;
#pragma unroll
            for (int i = 0; i < kDownWarps; ++i) h += part[i][threadIdx.x];
            sums[threadIdx.x] = h;
        }
        cluster_sync();
        if (rank == 0) {
            float v[kCluster], h = 0.0f;
#pragma unroll
            for (int i = 0; i < kCluster; ++i) v[i] = cluster_load(&sums[threadIdx.x], i);
#pragma unroll
            for (int i = 0; i < kCluster; ++i) h += v[i];
            h *= scale;
            const int j = j0 + threadIdx.x / 16, t = nth_token(mask, threadIdx.x % 16);
            if (t >= 0 && j < p.R) {
                const uint32_t hi = dev::f32_to_bf16_rne(h);
                const float top = __uint_as_float(hi << 16);
                p.h[(int64_t)t * p.R + j] = (uint16_t)hi;
                // beside an infinity (or a NaN) nothing: inf - inf is not its rest
                p.h[(int64_t)(p.M + t) * p.R + j] =
                    isfinite(top) ? (uint16_t)dev::f32_to_bf16_rne(h - top) : (uint16_t)0;
            }
        }
        cluster_sync();                                      // sums have been read
        mask = drop_tokens(mask, 16);
    }
}

}  // namespace

size_t lora_scratch_bytes(int64_t M) {
    return (size_t)(2 * M * kLoraMaxRank * 2 + 255) & ~(size_t)255;
}

qz_status launch_lora(const void *a, const void *lora_a, const void *lora_b, const void *adapters,
                      const void *lora_scales, int64_t n_adapters, int64_t rank, int64_t M,
                      int64_t K, void *scratch, LoraUp *up, cudaStream_t st) {
    LoraArgs p{};
    p.a = static_cast<const uint16_t *>(a);
    p.down = static_cast<const uint16_t *>(lora_a);
    p.ids = static_cast<const int32_t *>(adapters);
    p.scales = static_cast<const float *>(lora_scales);
    p.M = (int)M; p.K = (int)K; p.R = (int)rank; p.adapters = (int)n_adapters;
    p.h = static_cast<uint16_t *>(scratch);
    p.err_word = device_error_word();
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    *up = LoraUp{static_cast<const uint16_t *>(lora_b), p.h, p.ids, p.R, p.adapters};
    const unsigned used = (unsigned)(M < n_adapters ? M : n_adapters);
    lora_down_kernel<<<dim3(used, (unsigned)ceil_div(rank, 16), kCluster), 32 * kDownWarps, 0, st>>>(p);
    return launch_status();
}

}  // namespace qz
