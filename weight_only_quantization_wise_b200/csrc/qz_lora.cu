// qz_lora.cu -- low-rank adapters of many requests beside a packed projection:
//   y_m = bf16( sum_k a_mk w^_nk + s_r sum_j B_r[n][j] h_mj ),  h_mj = sum_k A_r[j][k] a_mk,
// r the adapter of token m.  Two kernels make the second term, an M x N fp32
// array that the GEMV's sums start from (qz_gemv.cu, ADD), so the output is
// rounded once.
//
// Tokens that share an adapter are worked on together, so each adapter in use
// is read once: every block finds the tokens of its adapter from the M
// indices itself (at most 64).  Both products run on mma.sync m16n8k16 with
// bf16 operands and fp32 sums: 16 ranks (or rows of B) x 8 tokens.  The
// fragments' k order is free as long as both operands agree, so a lane reads
// 16 consecutive bytes of a row: k = 8 tid .. 8 tid + 7 of every 32.
//   down:   one block per (adapter in use, 16 ranks); its 16 warps share K and
//           their sums meet in shared memory in a fixed order.  h is kept as
//           two bf16 values, h = hi + lo (2^-17 of h), the operands of the
//           second product.
//   up:     a warp per 16 rows of B, for all adapters in use.
#include <cuda_runtime.h>

#include "qz_internal.cuh"

namespace qz {
namespace {

constexpr int kMaxTokens = 64;
constexpr unsigned kErrIndex = 2u;     // bit of the device error word: adapter index out of range
constexpr int kDownWarps = 16;
constexpr int kUpWarps = 4;

struct LoraArgs {
    const uint16_t *a, *down, *up;     // M x K; adapters x R x K; adapters x N x R
    const int32_t *ids;
    const float *scales;
    int M, N, K, R, adapters;
    uint16_t *h;                       // [2][M][R]: hi, lo
    float *delta;                      // M x N
    unsigned int *err_word;
};

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Adapter of token m, -1 for none (or an index out of range).
__device__ __forceinline__ int adapter_of(const LoraArgs &p, int m) {
    const int id = p.ids[m];
    return id >= 0 && id < p.adapters ? id : -1;
}

// Tokens whose adapter is `id`, as a bit mask (all lanes of a warp).
__device__ __forceinline__ uint64_t tokens_of(const LoraArgs &p, int id, int lane) {
    const uint32_t lo = __ballot_sync(0xFFFFFFFFu, lane < p.M && adapter_of(p, lane) == id);
    const uint32_t hi =
        __ballot_sync(0xFFFFFFFFu, lane + 32 < p.M && adapter_of(p, lane + 32) == id);
    return (uint64_t)hi << 32 | lo;
}

// The c-th lowest token of the mask, -1 when there are fewer.
__device__ __forceinline__ int nth_token(uint64_t mask, int c) {
    for (int i = 0; i < c; ++i) mask &= mask - 1;
    return mask ? __ffsll((long long)mask) - 1 : -1;
}

// ---------------------------------------------------------------------------
// down: grid (M, ceil(R / 16)); block m works when token m is the first of its adapter
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(32 * kDownWarps) lora_down_kernel(const LoraArgs p) {
    grid_release();
    __shared__ float part[kDownWarps][16 * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
    const int m = blockIdx.x, j0 = 16 * blockIdx.y;
    const int raw = p.ids[m];
    if (raw >= p.adapters && threadIdx.x == 0 && j0 == 0) atomicOr(p.err_word, kErrIndex);
    const int id = adapter_of(p, m);
    if (id < 0) return;
    uint64_t mask = tokens_of(p, id, lane);
    if (__ffsll((long long)mask) - 1 != m) return;
    const float scale = p.scales[id];
    const uint16_t *row0 = p.down + ((int64_t)id * p.R + j0 + gid) * p.K + 8 * tid;
    const uint16_t *row1 = row0 + (int64_t)8 * p.K;
    const bool v0 = j0 + gid < p.R, v1 = j0 + gid + 8 < p.R;
    const int steps = p.K / 32;                              // K is a multiple of 128
    const int s0 = warp * steps / kDownWarps, s1 = (warp + 1) * steps / kDownWarps;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    while (mask) {
        const int tok = nth_token(mask, gid);                // column gid
        const uint16_t *act = p.a + (int64_t)(tok < 0 ? 0 : tok) * p.K + 8 * tid;
        float acc[2][4] = {};
#pragma unroll 4
        for (int s = s0; s < s1; ++s) {
            const uint4 x = v0 ? dev::ld_stream_v4(row0 + 32 * s) : none;
            const uint4 y = v1 ? dev::ld_stream_v4(row1 + 32 * s) : none;
            const uint4 b = tok >= 0 ? __ldg(reinterpret_cast<const uint4 *>(act + 32 * s)) : none;
            dev::mma_bf16_16816(acc[0], x.x, y.x, x.y, y.y, b.x, b.y);
            dev::mma_bf16_16816(acc[1], x.z, y.z, x.w, y.w, b.z, b.w);
        }
        // acc[.][i]: rank gid + 8 (i >> 1), token column 2 tid + (i & 1)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            part[warp][(gid + 8 * (i >> 1)) * 8 + 2 * tid + (i & 1)] = acc[0][i] + acc[1][i];
        __syncthreads();
        if (threadIdx.x < 128) {
            float h = 0.0f;
            for (int w = 0; w < kDownWarps; ++w) h += part[w][threadIdx.x];
            h *= scale;
            const int j = j0 + threadIdx.x / 8, t = nth_token(mask, threadIdx.x % 8);
            if (t >= 0 && j < p.R) {
                const uint32_t hi = dev::f32_to_bf16_rne(h);
                p.h[(int64_t)t * p.R + j] = (uint16_t)hi;
                p.h[(int64_t)(p.M + t) * p.R + j] =
                    (uint16_t)dev::f32_to_bf16_rne(h - __uint_as_float(hi << 16));
            }
        }
        __syncthreads();
        for (int i = 0; i < 8 && mask; ++i) mask &= mask - 1;
    }
}

// ---------------------------------------------------------------------------
// up: a warp per 16 rows of B
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(32 * kUpWarps) lora_up_kernel(const LoraArgs p) {
    grid_release();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gid = lane >> 2, tid = lane & 3;
    const int n0 = 16 * (blockIdx.x * kUpWarps + warp);
    if (n0 >= p.N) return;
    const int ra = n0 + gid, rb = ra + 8;
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    uint64_t todo = p.M == 64 ? ~0ull : (1ull << p.M) - 1;
    grid_wait();                                             // h, and the buffer delta lies in
    while (todo) {
        const int first = __ffsll((long long)todo) - 1;
        const int id = adapter_of(p, first);
        uint64_t mask = tokens_of(p, id, lane);
        todo &= ~mask;
        const uint16_t *row0 = p.up + ((int64_t)(id < 0 ? 0 : id) * p.N + ra) * p.R + 8 * tid;
        while (mask) {
            const int tok = nth_token(mask, gid);            // column gid
            float acc[4] = {};
            if (id >= 0) {
                for (int j = 0; j < p.R; j += 32) {
                    const bool in = j + 8 * tid < p.R;       // R is a multiple of 8
                    const uint4 x = in && ra < p.N ? dev::ld_stream_v4(row0 + j) : none;
                    const uint4 y = in && rb < p.N ? dev::ld_stream_v4(row0 + (int64_t)8 * p.R + j) : none;
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint4 b =
                            in && tok >= 0
                                ? __ldcg(reinterpret_cast<const uint4 *>(
                                      p.h + (int64_t)(part * p.M + tok) * p.R + j + 8 * tid))
                                : none;
                        dev::mma_bf16_16816(acc, x.x, y.x, x.y, y.y, b.x, b.y);
                        dev::mma_bf16_16816(acc, x.z, y.z, x.w, y.w, b.z, b.w);
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = nth_token(mask, 2 * tid + (i & 1)), n = i < 2 ? ra : rb;
                if (t >= 0 && n < p.N) __stcg(p.delta + (int64_t)t * p.N + n, acc[i]);
            }
            for (int i = 0; i < 8 && mask; ++i) mask &= mask - 1;
        }
    }
}

size_t h_bytes(int64_t M) { return (size_t)(2 * M * kLoraMaxRank * 2 + 255) & ~(size_t)255; }

}  // namespace

size_t lora_scratch_bytes(int64_t M, int64_t N) { return h_bytes(M) + (size_t)M * N * sizeof(float); }

qz_status launch_lora(const void *a, const void *lora_a, const void *lora_b, const void *adapters,
                      const void *lora_scales, int64_t n_adapters, int64_t rank, int64_t M,
                      int64_t N, int64_t K, void *scratch, const float **delta, cudaStream_t st) {
    LoraArgs p{};
    p.a = static_cast<const uint16_t *>(a);
    p.down = static_cast<const uint16_t *>(lora_a);
    p.up = static_cast<const uint16_t *>(lora_b);
    p.ids = static_cast<const int32_t *>(adapters);
    p.scales = static_cast<const float *>(lora_scales);
    p.M = (int)M; p.N = (int)N; p.K = (int)K; p.R = (int)rank; p.adapters = (int)n_adapters;
    p.h = static_cast<uint16_t *>(scratch);
    p.delta = reinterpret_cast<float *>(static_cast<char *>(scratch) + h_bytes(M));
    p.err_word = device_error_word();
    if (p.err_word == nullptr) return QZ_ERR_CUDA;
    *delta = p.delta;
    lora_down_kernel<<<dim3((unsigned)M, (unsigned)ceil_div(rank, 16)), 32 * kDownWarps, 0, st>>>(p);
    const qz_status s = launch_status();
    if (s != QZ_OK) return s;
    // the up kernel may start while the down kernel finishes; it waits for it
    // before it reads h
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div(N, 16 * kUpWarps));
    cfg.blockDim = dim3(32 * kUpWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, lora_up_kernel, p);
    return launch_status();
}

}  // namespace qz
