// kv_pages.cu -- writing the paged 4-bit KV cache (include/strata_attn.h):
// rotary + encoder of new rows into their slots, and copies of whole pages.
#include <cstring>
#include <new>
#include <type_traits>

#include "abi_internal.h"
#include "kv4_row.cuh"

using namespace strata;

strata_status strata_check_kv4_cache(const strata_kv4_cache *c) {
    if (!c) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL cache");
    if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
        return strata_set_error(STRATA_ERR_UNSUPPORTED, "head_dim %d not in {64, 128, 256}", c->head_dim);
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return strata_set_error(STRATA_ERR_UNSUPPORTED, "page_size %d is not a power of two in 16..1024", c->page_size);
    if (c->n_kv_heads < 1 || c->n_pages < 0)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "n_kv_heads %d, n_pages %lld", c->n_kv_heads, (long long)c->n_pages);
    if (c->n_pages > (int64_t)0xfffffffe / c->page_size / c->n_kv_heads)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "the cache has 2^32 - 1 rows or more");
    const void *p[4] = {c->k_codes, c->k_scales, c->v_codes, c->v_scales};
    for (int i = 0; i < 4; ++i) {
        if (!p[i] && c->n_pages > 0) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL plane of a cache");
        if (reinterpret_cast<uintptr_t>(p[i]) & 15)
            return strata_set_error(STRATA_ERR_INVALID_ARG, "the planes of a cache must be 16-byte aligned");
    }
    return STRATA_OK;
}

namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ append
// Row layout of the codec's encoder (its bits depend on the butterflies'
// order, strides 1, 2, ..., D/2): a row is spread over D / (8 R) lanes, lane l
// holding values 8 (l + m D / (8 R)) + e, m < R runs of e < 8.
template <int D>
struct Row {
    static constexpr int kRuns = D == 64 ? 2 : 4;
    static constexpr int kLanes = D / (8 * kRuns);
};

// two values at a time (add and fused multiply-add of pairs); a - b is
// fma(b, -1, a), which rounds the same
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <int D>
__device__ __forceinline__ void fwht_ordered(float (&x)[Row<D>::kRuns][8], int l) {
    using R = Row<D>;
    uint64_t p[R::kRuns][4];
    const uint64_t minus = pair_of(-1.f, -1.f);
#pragma unroll
    for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) p[m][e] = pair_of(__fadd_rn(x[m][2 * e], x[m][2 * e + 1]), __fsub_rn(x[m][2 * e], x[m][2 * e + 1]));
#pragma unroll
    for (int s = 1; s < 4; s <<= 1)
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!(e & s)) {
                    const uint64_t a = p[m][e], b = p[m][e + s];
                    p[m][e] = add_pair(a, b);
                    p[m][e + s] = fma_pair(b, minus, a);
                }
#pragma unroll
    for (int k = 1; k < R::kLanes; k <<= 1) {
        const float sg = (l & k) ? -1.f : 1.f;  // the upper lane forms partner - own
        const uint64_t sg2 = pair_of(sg, sg);
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float a, b;
                split(p[m][e], a, b);
                const uint64_t o = pair_of(__shfl_xor_sync(kFullMask, a, k), __shfl_xor_sync(kFullMask, b, k));
                p[m][e] = fma_pair(sg2, p[m][e], o);
            }
    }
#pragma unroll
    for (int s = 1; s < R::kRuns; s <<= 1)
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m)
            if (!(m & s))
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint64_t a = p[m][e], b = p[m + s][e];
                    p[m][e] = add_pair(a, b);
                    p[m + s][e] = fma_pair(b, minus, a);
                }
#pragma unroll
    for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) split(p[m][e], x[m][2 * e], x[m][2 * e + 1]);
}

struct AppendArgs {
    strata_kv4_cache c;
    const __nv_bfloat16 *k, *v;
    int64_t k_tok, v_tok;
    const int32_t *positions;
    const int64_t *slots;
    int64_t n_tokens;
    int tokens_per_block;
};

// What turns a key row: nothing, or pairs that one lane holds (the half layout
// over the whole head: a chunk's partner is R / 2 runs on; the interleaved one),
// or partners read once more from memory, in whole chunks or one by one
enum { kPlain, kHalfWhole, kInterleaved, kHalfChunks, kOther };

// One block takes tokens_per_block tokens: their cosines and sines once
// (fp64) into shared memory, while the first rows are on their way, then the key
// rows and the value rows of each (in this order, so that warps agree). Values
// go in pairs where the operation has a form for two. Measured: 8,192 tokens of
// 4 heads of 128 14.4 us (1.5 TB/s, 35 instructions a value, issue active 65 %),
// without rotary 11.7 us; 64 tokens 7.7 us a call, the call's own cost. Exact
// rounding is not what bounds it: strata_kv4_encode, with the same bits, takes
// 8.6 us for these rows. It divides once a lane instead of once a run, skips the
// clamp for normal scales and packs codes by byte permutes, none of which is
// done here, beside this kernel's divisions by the page and the heads. At 64
// registers and 4 blocks for an SM: 16.5 us.
template <int D, int MODE>
__global__ void __launch_bounds__(kThreads) k_kv4_append(const __grid_constant__ RopeTable tab,
                                                        const __grid_constant__ AppendArgs a) {
    using R = Row<D>;
    extern __shared__ __align__(16) float2 cs[];  // [tokens_per_block][rd / 2]
    const int pairs = tab.rd / 2;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_block;
    const int nt = (int)min((int64_t)a.tokens_per_block, a.n_tokens - t0);
    const int heads = a.c.n_kv_heads;
    const int k_rows = nt * heads, rows = 2 * k_rows;
    const int l = threadIdx.x % R::kLanes;
    constexpr int kRowsPerPass = kThreads / R::kLanes;
    int r = threadIdx.x / R::kLanes;
    uint4 raw[R::kRuns];
    int64_t slot = -1;
    const __nv_bfloat16 *src = nullptr;
    int t = 0, h = 0;
    auto fetch = [&]() {
        if (r >= rows) return;
        const int q = r < k_rows ? r : r - k_rows;
        t = q / heads;
        h = q - t * heads;
        src = (r < k_rows ? a.k + (t0 + t) * a.k_tok : a.v + (t0 + t) * a.v_tok) + (int64_t)h * D;
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m) raw[m] = *reinterpret_cast<const uint4 *>(src + 8 * (l + R::kLanes * m));
        slot = a.slots[t0 + t];
    };
    fetch();
    if (MODE != kPlain) {
        for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
            const int u = i / pairs;
            cs[i] = rope_cs(tab, i - u * pairs, a.positions[t0 + u]);
        }
        __syncthreads();
    }
    for (int r0 = 0; r0 < rows; r0 += kRowsPerPass) {  // block-uniform: the shuffles need whole warps
        const bool live = r < rows, is_v = r >= k_rows;
        float x[R::kRuns][8];
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m) {
            const uint32_t w[4] = {raw[m].x, raw[m].y, raw[m].z, raw[m].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[m][2 * j] = live ? bf16_lo(w[j]) : 0.f;
                x[m][2 * j + 1] = live ? bf16_hi(w[j]) : 0.f;
            }
        }
        if (MODE != kPlain && live && !is_v) {
            const float2 *ct = cs + t * pairs;
            if constexpr (MODE == kHalfWhole) {
#pragma unroll
                for (int m = 0; m < R::kRuns / 2; ++m) {
                    const float4 *c = reinterpret_cast<const float4 *>(ct + 8 * (l + R::kLanes * m));
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 k = c[e / 2];
                        const float2 c0 = make_float2(k.x, k.y), c1 = make_float2(k.z, k.w);
                        float *u = x[m] + e, *v = x[m + R::kRuns / 2] + e;
                        const uint32_t ru = pack_bf16(rope_first(u[0], v[0], c0), rope_first(u[1], v[1], c1));
                        const uint32_t rv = pack_bf16(rope_second(u[0], v[0], c0), rope_second(u[1], v[1], c1));
                        u[0] = bf16_lo(ru), u[1] = bf16_hi(ru), v[0] = bf16_lo(rv), v[1] = bf16_hi(rv);
                    }
                }
            } else if constexpr (MODE == kInterleaved) {
#pragma unroll
                for (int m = 0; m < R::kRuns; ++m) {
                    const int c8 = 8 * (l + R::kLanes * m);
                    if (c8 >= tab.rd) continue;
                    const float4 *c = reinterpret_cast<const float4 *>(ct + c8 / 2);
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 k = c[e / 4];
                        const float2 c0 = make_float2(k.x, k.y), c1 = make_float2(k.z, k.w);
                        float *u = x[m] + e;
                        const uint32_t r0_ = pack_bf16(rope_first(u[0], u[1], c0), rope_second(u[0], u[1], c0));
                        const uint32_t r1_ = pack_bf16(rope_first(u[2], u[3], c1), rope_second(u[2], u[3], c1));
                        u[0] = bf16_lo(r0_), u[1] = bf16_hi(r0_), u[2] = bf16_lo(r1_), u[3] = bf16_hi(r1_);
                    }
                }
            } else if constexpr (MODE == kHalfChunks) {
#pragma unroll
                for (int m = 0; m < R::kRuns; ++m) {
                    const int c8 = 8 * (l + R::kLanes * m);
                    if (c8 >= tab.rd) continue;
                    const bool second = c8 >= pairs;
                    const uint4 q4 = *reinterpret_cast<const uint4 *>(src + (second ? c8 - pairs : c8 + pairs));
                    const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
                    const float4 *c = reinterpret_cast<const float4 *>(ct + (second ? c8 - pairs : c8));
                    const float sg = second ? 1.f : -1.f;  // u c - v s, v c + u s: a negated product rounds the same
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 k = c[e / 2];
                        float *u = x[m] + e;
                        const uint32_t w = pack_bf16(__fadd_rn(__fmul_rn(u[0], k.x), sg * __fmul_rn(bf16_lo(q[e / 2]), k.y)),
                                                     __fadd_rn(__fmul_rn(u[1], k.z), sg * __fmul_rn(bf16_hi(q[e / 2]), k.w)));
                        u[0] = bf16_lo(w), u[1] = bf16_hi(w);
                    }
                }
            } else {
#pragma unroll
                for (int m = 0; m < R::kRuns; ++m) {
                    const int c8 = 8 * (l + R::kLanes * m);  // first value of the chunk
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i = c8 + e;
                        if (i < tab.rd) {
                            const float p = __bfloat162float(src[rope_partner(tab, i)]);
                            const float2 c = ct[rope_pair(tab, i)];
                            const float y = rope_is_second(tab, i) ? rope_second(p, x[m][e], c) : rope_first(x[m][e], p, c);
                            x[m][e] = __bfloat162float(__float2bfloat16_rn(y));
                        }
                    }
                }
            }
        }
        const int64_t page = slot / a.c.page_size;
        const bool store = live && slot >= 0 && page < a.c.n_pages;
        const int64_t row = (page * heads + h) * a.c.page_size + (slot - page * a.c.page_size);
        uint32_t *codes = static_cast<uint32_t *>(is_v ? a.c.v_codes : a.c.k_codes) + (store ? row * (D / 8) : 0);
        __half *scales = static_cast<__half *>(is_v ? a.c.v_scales : a.c.k_scales) + (store ? row * (D / 32) : 0);
        r += kRowsPerPass;
        fetch();  // the next row, behind this one's arithmetic
        fwht_ordered<D>(x, l);
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m) {
            float amax = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[m][e] = __fmul_rn(x[m][e], rsqrt_dim<D>());
                amax = fmaxf(amax, fabsf(x[m][e]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(kFullMask, amax, 2));
            const __half hs = __float2half_rn(fminf(__fdiv_rn(amax, 7.f), 65504.f));
            const float s = __half2float(hs);
            const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
            // 1.5 * 2^23 + 8 rounds the exact product to an integer, ties to even, and
            // leaves q + 8 in the low bits; a quotient of 8 or more (tiny or saturated
            // scales) ends at 7 like any other
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float q = fminf(fmaxf(__fmaf_rn(x[m][e], inv, 12582920.f), 12582913.f), 12582927.f);
                word |= (__float_as_uint(q) & 15u) << (4 * e);
            }
            if (store) {
                const int chunk = l + R::kLanes * m;
                codes[chunk] = word;
                if ((l & 3) == 0) scales[chunk / 4] = hs;
            }
        }
    }
}

// ------------------------------------------------------------- copy of pages
constexpr int kCopyCaches = 64;
constexpr int kCopyPairs = 2000;

// The lists travel by value in the launch's parameters: no device copy of
// them, nothing to free, and a captured graph keeps them.
template <int PAIRS>
struct CopyArgs {
    void *plane[kCopyCaches][4];
    uint32_t src[PAIRS], dst[PAIRS];
    int n_caches, n_pairs;
    uint32_t code_vecs, scale_vecs;  // 16-byte words of a page in a code / scale plane
};

// Bound by HBM: 400 pages of 37 KB in 48 caches 239 us (5.9 TB/s of 2 x 708 MB),
// 8 pages 7.8 us a call.
template <int PAIRS>
__global__ void __launch_bounds__(kThreads) k_kv4_copy(const __grid_constant__ CopyArgs<PAIRS> a) {
    const int64_t n = (int64_t)a.n_caches * a.n_pairs * 4;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const int plane = (int)(i & 3);
        const int64_t cp = i >> 2;
        const int cache = (int)(cp / a.n_pairs), pair = (int)(cp - (int64_t)cache * a.n_pairs);
        const uint32_t vecs = (plane & 1) ? a.scale_vecs : a.code_vecs;
        uint4 *base = static_cast<uint4 *>(a.plane[cache][plane]);
        const uint4 *s = base + (int64_t)a.src[pair] * vecs;
        uint4 *d = base + (int64_t)a.dst[pair] * vecs;
        for (uint32_t j = threadIdx.x; j < vecs; j += kThreads) d[j] = s[j];
    }
}

template <int PAIRS>
cudaError_t launch_copy(const strata_kv4_cache *caches, int n_caches, const int32_t *src, const int32_t *dst, int n,
                        cudaStream_t st) {
    static_assert(sizeof(CopyArgs<PAIRS>) <= 32000, "kernel parameters");
    CopyArgs<PAIRS> a;
    for (int c = 0; c < n_caches; ++c) {
        a.plane[c][0] = caches[c].k_codes;
        a.plane[c][1] = caches[c].k_scales;
        a.plane[c][2] = caches[c].v_codes;
        a.plane[c][3] = caches[c].v_scales;
    }
    for (int i = 0; i < n; ++i) {
        a.src[i] = (uint32_t)src[i];
        a.dst[i] = (uint32_t)dst[i];
    }
    a.n_caches = n_caches;
    a.n_pairs = n;
    const uint32_t rows = (uint32_t)(caches[0].n_kv_heads * caches[0].page_size);
    a.code_vecs = rows * (uint32_t)(caches[0].head_dim / 32);
    a.scale_vecs = rows * (uint32_t)(caches[0].head_dim / 16) / 16;
    const int64_t units = (int64_t)n_caches * n * 4;
    k_kv4_copy<PAIRS><<<(int)(units < 4096 ? units : 4096), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

// The pages named so far, open addressing: bit 0 source, bit 1 destination.
struct PageSet {
    int64_t cap;
    int32_t *page;  // -1: empty
    uint8_t *mark;
    uint8_t &at(int32_t p) {
        uint64_t i = ((uint64_t)(uint32_t)p * 0x9E3779B97F4A7C15ull) >> 20 & (uint64_t)(cap - 1);
        while (page[i] != -1 && page[i] != p) i = (i + 1) & (uint64_t)(cap - 1);
        if (page[i] == -1) page[i] = p, mark[i] = 0;
        return mark[i];
    }
};

}  // namespace

extern "C" strata_status strata_kv4_append(const strata_kv4_cache *cache, strata_rope rope, const void *k,
                                           int64_t k_token_stride, const void *v, int64_t v_token_stride,
                                           const int32_t *positions, const int64_t *slots, int64_t n_tokens,
                                           strata_stream_t stream) {
    const strata_status s = strata_check_kv4_cache(cache);
    if (s != STRATA_OK) return s;
    if (n_tokens < 0) return strata_set_error(STRATA_ERR_INVALID_ARG, "n_tokens %lld < 0", (long long)n_tokens);
    if (rope && rope->desc.head_dim != cache->head_dim)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "the rotary handle has head_dim %d, the cache %d",
                                rope->desc.head_dim, cache->head_dim);
    if (n_tokens == 0) return STRATA_OK;
    if (!k || !v || !slots || (rope && !positions))
        return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) ||
        (reinterpret_cast<uintptr_t>(slots) & 7) || (reinterpret_cast<uintptr_t>(positions) & 3))
        return strata_set_error(STRATA_ERR_INVALID_ARG, "k and v must be 16-byte, slots 8-byte, positions 4-byte aligned");
    const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
    if (((k_token_stride | v_token_stride) & 7) || (n_tokens > 1 && (k_token_stride < row || v_token_stride < row)))
        return strata_set_error(STRATA_ERR_INVALID_ARG,
                                "token strides must be multiples of 8 elements and hold the heads of a token");
    static const RopeTable none = {};
    const RopeTable &tab = rope ? rope->table : none;
    AppendArgs a{*cache, static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(v),
                 k_token_stride, v_token_stride, positions, slots, n_tokens, 1};
    // whole blocks of rows, but no more tokens than leave every SM a block
    const int lanes = cache->head_dim == 256 ? 8 : 4;
    int64_t tpb = kThreads / lanes / (2 * (int64_t)cache->n_kv_heads);
    const int64_t spread = (n_tokens + 147) / 148;
    tpb = tpb < 1 ? 1 : tpb;
    tpb = tpb > spread ? spread : tpb;
    tpb = tpb > 32 ? 32 : tpb;
    a.tokens_per_block = (int)tpb;
    const int64_t grid = (n_tokens + tpb - 1) / tpb;
    if (grid > 0x7fffffff) return strata_set_error(STRATA_ERR_INVALID_ARG, "n_tokens %lld", (long long)n_tokens);
    const size_t smem = (size_t)tpb * (tab.rd / 2) * sizeof(float2);
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int mode = tab.rd == 0                                    ? kPlain
                     : tab.half && tab.rd == cache->head_dim ? kHalfWhole
                     : !tab.half && tab.rd % 8 == 0          ? kInterleaved
                     : tab.half && tab.rd % 16 == 0          ? kHalfChunks
                                                             : kOther;
    auto launch = [&](auto dim) {
        constexpr int D = decltype(dim)::value;
        if (mode == kPlain)
            k_kv4_append<D, kPlain><<<(int)grid, kThreads, 0, st>>>(tab, a);
        else if (mode == kHalfWhole)
            k_kv4_append<D, kHalfWhole><<<(int)grid, kThreads, smem, st>>>(tab, a);
        else if (mode == kInterleaved)
            k_kv4_append<D, kInterleaved><<<(int)grid, kThreads, smem, st>>>(tab, a);
        else if (mode == kHalfChunks)
            k_kv4_append<D, kHalfChunks><<<(int)grid, kThreads, smem, st>>>(tab, a);
        else
            k_kv4_append<D, kOther><<<(int)grid, kThreads, smem, st>>>(tab, a);
    };
    if (cache->head_dim == 64)
        launch(std::integral_constant<int, 64>{});
    else if (cache->head_dim == 128)
        launch(std::integral_constant<int, 128>{});
    else
        launch(std::integral_constant<int, 256>{});
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return strata_set_error(STRATA_ERR_CUDA, "kv4 append launch: %s", cudaGetErrorString(e));
    return STRATA_OK;
}

extern "C" strata_status strata_kv4_copy_pages(const strata_kv4_cache *caches, int32_t n_caches, const int32_t *src,
                                               const int32_t *dst, int64_t n_pairs, strata_stream_t stream) {
    if (n_caches < 0 || n_pairs < 0)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "n_caches %d, n_pairs %lld", n_caches, (long long)n_pairs);
    if (n_caches == 0 || n_pairs == 0) return STRATA_OK;
    if (!caches || !src || !dst) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL array");
    int64_t pages = INT64_MAX;
    for (int c = 0; c < n_caches; ++c) {
        const strata_status s = strata_check_kv4_cache(&caches[c]);
        if (s != STRATA_OK) return s;
        if (caches[c].head_dim != caches[0].head_dim || caches[c].page_size != caches[0].page_size ||
            caches[c].n_kv_heads != caches[0].n_kv_heads)
            return strata_set_error(STRATA_ERR_INVALID_ARG, "cache %d has another shape than cache 0", c);
        pages = caches[c].n_pages < pages ? caches[c].n_pages : pages;
    }
    if (n_pairs > pages) return strata_set_error(STRATA_ERR_INVALID_ARG, "more pairs than pages");
    PageSet set{64, nullptr, nullptr};
    while (set.cap < 4 * n_pairs) set.cap *= 2;
    set.page = new (std::nothrow) int32_t[set.cap];
    set.mark = new (std::nothrow) uint8_t[set.cap];
    strata_status s = STRATA_OK;
    if (!set.page || !set.mark) {
        s = strata_set_error(STRATA_ERR_OOM, "host memory of %lld pairs", (long long)n_pairs);
    } else {
        memset(set.page, 0xff, sizeof(int32_t) * (size_t)set.cap);
        for (int64_t i = 0; i < n_pairs && s == STRATA_OK; ++i) {
            if (src[i] < 0 || src[i] >= pages || dst[i] < 0 || dst[i] >= pages) {
                s = strata_set_error(STRATA_ERR_INVALID_ARG, "pair %lld: page %d -> %d of %lld", (long long)i, src[i],
                                     dst[i], (long long)pages);
                break;
            }
            uint8_t &a = set.at(src[i]);
            a |= 1;
            const bool clash = (a & 2) != 0;
            uint8_t &b = set.at(dst[i]);
            if (clash || b != 0)
                s = strata_set_error(STRATA_ERR_INVALID_ARG,
                                     "pair %lld: page %d -> %d: a destination is named twice or is a source too",
                                     (long long)i, src[i], dst[i]);
            b |= 2;
        }
    }
    delete[] set.page;
    delete[] set.mark;
    if (s != STRATA_OK) return s;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    for (int c = 0; c < n_caches; c += kCopyCaches) {
        const int nc = n_caches - c < kCopyCaches ? n_caches - c : kCopyCaches;
        for (int64_t i = 0; i < n_pairs; i += kCopyPairs) {
            const int n = (int)(n_pairs - i < kCopyPairs ? n_pairs - i : kCopyPairs);
            // short lists take a launch with few parameter bytes
            const cudaError_t e = n <= 64 ? launch_copy<64>(caches + c, nc, src + i, dst + i, n, st)
                                          : launch_copy<kCopyPairs>(caches + c, nc, src + i, dst + i, n, st);
            if (e != cudaSuccess) return strata_set_error(STRATA_ERR_CUDA, "page copy launch: %s", cudaGetErrorString(e));
        }
    }
    return STRATA_OK;
}
