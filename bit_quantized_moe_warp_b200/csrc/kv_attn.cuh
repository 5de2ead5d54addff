// kv_attn.cuh -- what the attention kernels over the paged 4-bit cache share:
// their arguments, the division of work over CTAs, and the kernel that joins
// partial results.
#pragma once

#include <atomic>
#include <cfloat>
#include <math.h>

#include "common.cuh"
#include "kv4_row.cuh"

namespace strata {

struct AttnArgs {
    strata_kv4_cache c;
    strata_kv4_attn_desc d;
    const int32_t *positions;
    const __nv_bfloat16 *q;
    const int32_t *q_offsets, *kv_lens, *table;
    __nv_bfloat16 *out;
    void *workspace;
    int group, page_shift;
    float scale_log2;  // scale * log2(e)
    uint64_t group_inv;  // 2^64 / group, rounded up (0 for 1)
};
// row / group for 0 <= row < 2^31: exact, since the rounding of group_inv adds
// less than 2^31 / 2^64 of the divisor's reciprocal
__device__ __forceinline__ int by_group(const AttnArgs &a, int row) {
    return a.group_inv ? (int)__umul64hi((uint64_t)(uint32_t)row, a.group_inv) : row;
}

// Row r of a KV head's query rows (token-major, the group's heads inside), in
// the rotated basis: back through the transform, divided by its sum, rounded
// once.
template <int D>
__device__ __forceinline__ void store_row(const AttnArgs &a, float (&v)[D / 32], float l, int64_t t0, int hk, int r,
                                          int lane) {
    constexpr int P = D / 32;
    const int i = by_group(a, r), h = hk * a.group + r - i * a.group;
    const float f = l > 0.f ? rsqrt_dim<D>() / l : 0.f;
    fwht_warp<D>(v, lane);
    uint32_t w[P / 2];
#pragma unroll
    for (int j = 0; j < P / 2; ++j) w[j] = pack_bf16(v[2 * j] * f, v[2 * j + 1] * f);
    uint8_t *dst = reinterpret_cast<uint8_t *>(a.out + (t0 + i) * a.d.out_token_stride + (int64_t)h * D + lane * P);
    if constexpr (P == 2) *reinterpret_cast<uint32_t *>(dst) = w[0];
    if constexpr (P == 4) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    if constexpr (P == 8) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A value that is the same in every lane, so that the compiler sees it is:
// branches on it need no reconvergence
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kFullMask, v, 0); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// total * i / n, rounded down: where run i of n starts
__device__ __forceinline__ int64_t run_start(int64_t total, int64_t i, int64_t n) {
    const uint64_t x = (uint64_t)total * (uint64_t)i;
    return ((x | (uint64_t)n) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)n) : (int64_t)(x / (uint64_t)n);
}

// A sequence: its first query row, query rows and cached tokens, in range
struct SeqBase {
    int64_t t0;
    int n, L;
};
__device__ __forceinline__ void load_seq(SeqBase &s, const AttnArgs &a, int b) {
    s.t0 = min(max((int64_t)a.q_offsets[b], (int64_t)0), a.d.n_tokens);
    s.n = (int)(min(max((int64_t)a.q_offsets[b + 1], s.t0), a.d.n_tokens) - s.t0);
    s.L = (int)min((int64_t)max(a.kv_lens[b], 0), (int64_t)a.d.max_pages << a.page_shift);
}

constexpr int kSms = 148;
constexpr int kSplitMaxCtas = 2 * kSms;

struct Span {  // what k_attn_join needs of the last piece of a CTA
    int parts;  // CTAs that share it, 0: none
    int slot;   // of the first one; 0 for the others
    int t0, rows, hk, row0;
    int pad[2];
};

// One block for each piece that several CTAs share and two of its query rows at
// a time: 8 warps over the parts of a row ([ROWS][D + 4] floats, M and l behind
// the values), each with a running maximum of its own, then over each other, in
// a fixed order. Bound by the latency of its two dependent loads, the span and
// the parts.
template <int D, int ROWS>
__global__ void __launch_bounds__(512) k_attn_join(const __grid_constant__ AttnArgs a) {
    constexpr int P = D / 32, PART = D + 4, BATCH = P == 8 ? 2 : 4;
    constexpr int WPR = 8, RPB = 16 / WPR;
    __shared__ float so[WPR][RPB][D], sl[WPR][RPB], sm[WPR][RPB];
    griddep_launch_dependents();
    griddep_wait();
    const Span sp = static_cast<const Span *>(a.workspace)[blockIdx.x];
    if (sp.parts == 0) return;
    const float *parts = reinterpret_cast<const float *>(static_cast<const Span *>(a.workspace) + kSplitMaxCtas);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wr = warp % RPB, wq = warp / RPB;
    for (int r0 = RPB * blockIdx.y; r0 < sp.rows; r0 += RPB * gridDim.y) {
        const int r = r0 + wr;
        const bool live = r < sp.rows;
        float v[P], sum = 0.f, m = -FLT_MAX;
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] = 0.f;
        for (int i0 = wq; i0 < sp.parts && live; i0 += WPR * BATCH) {
            float w[BATCH][P];
            float2 ml[BATCH];
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int i = i0 + WPR * k;
                ml[k] = make_float2(-FLT_MAX, 0.f);
#pragma unroll
                for (int j = 0; j < P; ++j) w[k][j] = 0.f;
                if (i >= sp.parts) continue;
                const float *p = parts + (int64_t)((blockIdx.x + i) * 2 + (i ? 0 : sp.slot)) * (ROWS * PART);
                auto at = [&](int d) { return p + r * PART + d; };
                ml[k] = *reinterpret_cast<const float2 *>(at(D));
                if constexpr (P == 2) *reinterpret_cast<float2 *>(w[k]) = *reinterpret_cast<const float2 *>(at(lane * P));
                if constexpr (P >= 4)
#pragma unroll
                    for (int j = 0; j < P; j += 4)
                        *reinterpret_cast<float4 *>(w[k] + j) = *reinterpret_cast<const float4 *>(at(lane * P + j));
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
            const float f = ex2(m - top);
            m = top;
            sum *= f;
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] *= f;
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const float g = ex2(ml[k].x - m);
                sum = fmaf(ml[k].y, g, sum);
#pragma unroll
                for (int j = 0; j < P; ++j) v[j] = fmaf(w[k][j], g, v[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < P; ++j) so[wq][wr][lane * P + j] = v[j];
        if (lane == 0) sl[wq][wr] = sum, sm[wq][wr] = m;
        __syncthreads();
        if (wq == 0) {
            float top = m;
#pragma unroll
            for (int w = 1; w < WPR; ++w) top = fmaxf(top, sm[w][wr]);
            const float f = ex2(m - top);
            sum *= f;
#pragma unroll
            for (int j = 0; j < P; ++j) v[j] *= f;
#pragma unroll
            for (int w = 1; w < WPR; ++w) {
                const float g = ex2(sm[w][wr] - top);
                sum = fmaf(sl[w][wr], g, sum);
#pragma unroll
                for (int j = 0; j < P; ++j) v[j] = fmaf(so[w][wr][lane * P + j], g, v[j]);
            }
        }
        if (wq == 0 && live) store_row<D>(a, v, sum, sp.t0, sp.hk, sp.row0 + r, lane);
        __syncthreads();
    }
}

// The same for parts in planes of four values over the rows, [D / 4 + 1][ROWS]
// float4: many rows of few parts. A thread adds up one float4 of a row, so that
// a warp's loads lie together; then a warp takes a row for the transform.
template <int D, int ROWS>
__global__ void __launch_bounds__(512) k_attn_join_planes(const __grid_constant__ AttnArgs a) {
    constexpr int P = D / 32, RPB = 2048 / D;  // rows of a block: one float4 for each thread
    __shared__ float so[RPB][D], sl[RPB];
    griddep_launch_dependents();
    griddep_wait();
    const Span sp = static_cast<const Span *>(a.workspace)[blockIdx.x];
    if (sp.parts == 0) return;
    const float4 *parts = reinterpret_cast<const float4 *>(static_cast<const Span *>(a.workspace) + kSplitMaxCtas);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tr = threadIdx.x % RPB, plane = threadIdx.x / RPB;
    for (int r0 = RPB * blockIdx.y; r0 < sp.rows; r0 += RPB * gridDim.y) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f, m = -FLT_MAX;
        const int r = min(r0 + tr, sp.rows - 1);
        for (int i0 = 0; i0 < sp.parts; i0 += 4) {
            float4 w[4], ml[4];
            float top = m;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                ml[k] = make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
                const int i = i0 + k;
                if (i >= sp.parts) continue;
                const float4 *p = parts + (int64_t)((blockIdx.x + i) * 2 + (i ? 0 : sp.slot)) * (ROWS * (D / 4 + 1)) + r;
                ml[k] = p[(D / 4) * ROWS];
                w[k] = p[plane * ROWS];
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) top = fmaxf(top, ml[k].x);
            const float f = ex2(m - top);
            m = top;
            sum *= f;
            v.x *= f, v.y *= f, v.z *= f, v.w *= f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float g = ex2(ml[k].x - m);
                sum = fmaf(ml[k].y, g, sum);
                v.x = fmaf(w[k].x, g, v.x), v.y = fmaf(w[k].y, g, v.y);
                v.z = fmaf(w[k].z, g, v.z), v.w = fmaf(w[k].w, g, v.w);
            }
        }
        *reinterpret_cast<float4 *>(&so[tr][plane * 4]) = v;
        if (plane == 0) sl[tr] = sum;
        __syncthreads();
        for (int k = warp; k < RPB && r0 + k < sp.rows; k += 16) {
            float x[P];
#pragma unroll
            for (int j = 0; j < P; ++j) x[j] = so[k][lane * P + j];
            store_row<D>(a, x, sl[k], sp.t0, sp.hk, sp.row0 + r0 + k, lane);
        }
        __syncthreads();
    }
}

// A launch that may come up before the kernel in front of it in the stream has
// ended: the kernels wait (griddep_wait) before they touch memory.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t st, const Args &...args) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Dynamic shared memory of a kernel, set once for each device: done has a bit each
template <typename Kernel>
cudaError_t allow_smem(Kernel *kernel, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int D, int ROWS, bool PLANES>
cudaError_t launch_join(const AttnArgs &a, int ctas, cudaStream_t st) {
    const int64_t rows = (int64_t)a.d.max_q_len * a.group;  // a hint only: a block takes more rows in turn
    constexpr int RPB = PLANES ? 2048 / D : 2;
    const unsigned y = rows < 1 ? 1 : rows < ROWS ? (unsigned)(rows + RPB - 1) / RPB : ROWS / RPB;
    if constexpr (PLANES)
        return launch_early(k_attn_join_planes<D, ROWS>, dim3(ctas, y), 512, 0, st, a);
    else
        return launch_early(k_attn_join<D, ROWS>, dim3(ctas, y), 512, 0, st, a);
}

// Many query rows (kv_attn_tiles.cu): bytes of its partial results, the launch, and
// the launch of the self test, in which a role of every `every`-th CTA stops
// arriving from its piece `piece` on
struct AttnStall {
    int role;  // 0 keys, 1 values, 2 weights, 3 query rows
    int every, piece;
};
size_t attn_tiles_part_bytes(int head_dim);
cudaError_t launch_attn_tiles(const RopeTable &tab, const AttnArgs &a, cudaStream_t st);
cudaError_t launch_attn_tiles_stalled(const RopeTable &tab, const AttnArgs &a, const AttnStall &stall, cudaStream_t st);

}  // namespace strata
