// kv_pages.cu -- writing the paged 4-bit KV cache (include/strata_attn.h):
// rotary + encoder of new rows into their slots, and copies of whole pages.
#include <cstring>
#include <new>

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

template <int D>
__device__ __forceinline__ void fwht_ordered(float (&x)[Row<D>::kRuns][8], int l) {
    using R = Row<D>;
#pragma unroll
    for (int s = 1; s < 8; s <<= 1)
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!(e & s)) {
                    const float a = x[m][e], b = x[m][e + s];
                    x[m][e] = __fadd_rn(a, b);
                    x[m][e + s] = __fsub_rn(a, b);
                }
#pragma unroll
    for (int k = 1; k < R::kLanes; k <<= 1) {
        const float sg = (l & k) ? -1.f : 1.f;  // the upper lane forms partner - own
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[m][e] = __fmaf_rn(sg, x[m][e], __shfl_xor_sync(kFullMask, x[m][e], k));
    }
#pragma unroll
    for (int s = 1; s < R::kRuns; s <<= 1)
#pragma unroll
        for (int m = 0; m < R::kRuns; ++m)
            if (!(m & s))
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a = x[m][e], b = x[m + s][e];
                    x[m][e] = __fadd_rn(a, b);
                    x[m + s][e] = __fsub_rn(a, b);
                }
}

struct AppendArgs {
    strata_kv4_cache c;
    const __nv_bfloat16 *k, *v;
    int64_t k_tok, v_tok;
    const int32_t *positions;
    const int64_t *slots;
    int64_t n_tokens;
    int tokens_per_block;
    int chunked;  // rotary pairs lie in whole 8-value chunks
};

// One block takes tokens_per_block tokens: their cosines and sines once
// (fp64) into shared memory, then the 2 n_kv_heads rows of each.
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv4_append(const __grid_constant__ RopeTable tab,
                                                        const __grid_constant__ AppendArgs a) {
    using R = Row<D>;
    extern __shared__ float2 cs[];  // [tokens_per_block][rd / 2]
    const int pairs = tab.rd / 2;
    const int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_block;
    const int nt = (int)min((int64_t)a.tokens_per_block, a.n_tokens - t0);
    for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
        const int t = i / pairs;
        cs[i] = rope_cs(tab, i - t * pairs, a.positions[t0 + t]);
    }
    __syncthreads();
    const int heads = a.c.n_kv_heads;
    const int rows = nt * 2 * heads;
    const int l = threadIdx.x % R::kLanes;
    constexpr int kRowsPerPass = kThreads / R::kLanes;
    for (int r0 = 0; r0 < rows; r0 += kRowsPerPass) {  // block-uniform: the shuffles need whole warps
        const int r = r0 + threadIdx.x / R::kLanes;
        const bool live = r < rows;
        const int t = live ? r / (2 * heads) : 0;
        const int kvh = r - t * 2 * heads;
        const bool is_v = kvh >= heads;
        const int h = is_v ? kvh - heads : kvh;
        float x[R::kRuns][8];
        if (live) {
            const __nv_bfloat16 *src =
                (is_v ? a.v + (t0 + t) * a.v_tok : a.k + (t0 + t) * a.k_tok) + (int64_t)h * D;
            const float2 *ct = cs + t * pairs;
            const int rd = is_v ? 0 : tab.rd;
#pragma unroll
            for (int m = 0; m < R::kRuns; ++m) {
                const int c8 = 8 * (l + R::kLanes * m);  // first value of the chunk
                const uint4 w4 = *reinterpret_cast<const uint4 *>(src + c8);
                const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[m][2 * j] = bf16_lo(w[j]);
                    x[m][2 * j + 1] = bf16_hi(w[j]);
                }
                if (c8 >= rd) continue;
                float p[8];  // rotary partners
                if (!tab.half) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = x[m][e ^ 1];
                } else if (a.chunked) {
                    const uint4 q4 = *reinterpret_cast<const uint4 *>(src + (c8 < pairs ? c8 + pairs : c8 - pairs));
                    const uint32_t q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        p[2 * j] = bf16_lo(q[j]);
                        p[2 * j + 1] = bf16_hi(q[j]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[e] = c8 + e < rd ? __bfloat162float(src[rope_partner(tab, c8 + e)]) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = c8 + e;
                    if (i < rd) {
                        const float2 c = ct[rope_pair(tab, i)];
                        const float y = rope_is_second(tab, i) ? rope_second(p[e], x[m][e], c)
                                                               : rope_first(x[m][e], p[e], c);
                        x[m][e] = __bfloat162float(__float2bfloat16_rn(y));
                    }
                }
            }
        } else {
#pragma unroll
            for (int m = 0; m < R::kRuns; ++m)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[m][e] = 0.f;
        }
        fwht_ordered<D>(x, l);
        int64_t slot = live ? a.slots[t0 + t] : -1;
        const int64_t page = slot / a.c.page_size;
        const bool store = slot >= 0 && page < a.c.n_pages;
        const int64_t row = (page * heads + h) * a.c.page_size + (slot - page * a.c.page_size);
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
            uint32_t word = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                int q;
                if (fabsf(__fmul_rn(x[m][e], inv)) >= 8.f) {
                    q = x[m][e] > 0.f ? 7 : -7;
                } else {  // 1.5 * 2^23 rounds the exact product to an integer, ties to even
                    q = (int)(__float_as_uint(__fmaf_rn(x[m][e], inv, 12582912.f)) - 0x4b400000u);
                    q = q > 7 ? 7 : (q < -7 ? -7 : q);
                }
                word |= (uint32_t)(q + 8) << (4 * e);
            }
            if (store) {
                const int chunk = l + R::kLanes * m;
                void *codes = is_v ? a.c.v_codes : a.c.k_codes, *scales = is_v ? a.c.v_scales : a.c.k_scales;
                static_cast<uint32_t *>(codes)[row * (D / 8) + chunk] = word;
                if ((l & 3) == 0) static_cast<__half *>(scales)[row * (D / 32) + chunk / 4] = hs;
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
                 k_token_stride, v_token_stride, positions, slots, n_tokens, 1, tab.rd % 16 == 0};
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
    if (cache->head_dim == 64)
        k_kv4_append<64><<<(int)grid, kThreads, smem, st>>>(tab, a);
    else if (cache->head_dim == 128)
        k_kv4_append<128><<<(int)grid, kThreads, smem, st>>>(tab, a);
    else
        k_kv4_append<256><<<(int)grid, kThreads, smem, st>>>(tab, a);
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
