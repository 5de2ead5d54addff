// kv_attention.cu -- attention over the paged 4-bit KV cache
// (include/strata_attn.h).
//
// H is symmetric and orthonormal up to sqrt(D), so q . k' = (H q / sqrt D) . y
// for the stored row y = (c - 8) s, and sum_j p_j v'_j = H (sum_j p_j y_j) / sqrt D:
// a query row is rotated once on the way in and its output once on the way
// out, and the cache's rows are used as they are stored.
#include <cmath>

#include "abi_internal.h"
#include "kv4_row.cuh"

using namespace strata;

namespace {

struct AttnArgs {
    strata_kv4_cache c;
    strata_kv4_attn_desc d;
    const int32_t *positions;
    const __nv_bfloat16 *q;
    const int32_t *q_offsets, *kv_lens, *table;
    __nv_bfloat16 *out;
    int group, page_shift;
    float scale_log2;  // scale * log2(e)
};

// One warp per (token, query head): every key in turn, running maximum and
// sum of the softmax in registers.
template <int D>
__global__ void __launch_bounds__(128) k_attn_rows(const __grid_constant__ RopeTable tab,
                                                  const __grid_constant__ AttnArgs a) {
    constexpr int P = D / 32;
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
    const int b = blockIdx.z;
    if (h >= a.d.n_q_heads) return;
    const int64_t n_tok = a.d.n_tokens;
    const int64_t t0 = min(max((int64_t)a.q_offsets[b], (int64_t)0), n_tok);
    const int64_t t1 = min(max((int64_t)a.q_offsets[b + 1], t0), n_tok);
    const int L = (int)min((int64_t)max(a.kv_lens[b], 0), (int64_t)a.d.max_pages << a.page_shift);
    const int hk = h / a.group;
    for (int64_t t = t0 + blockIdx.x; t < t1; t += gridDim.x) {
        float q[P], o[P];
        load_query_row<D>(q, a.q + t * a.d.q_token_stride + (int64_t)h * D, tab, tab.rd ? a.positions[t] : 0,
                          a.scale_log2, lane);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = 0.f;
        const int64_t p = L - (t1 - t0) + (t - t0);
        const int64_t lo = a.d.window > 0 ? max((int64_t)0, p - a.d.window + 1) : 0;
        const int64_t hi = min((int64_t)L, p + 1);
        float m = -INFINITY, l = 0.f;
        for (int64_t j = lo; j < hi; ++j) {
            const int page = a.table[(int64_t)b * a.d.max_pages + (j >> a.page_shift)];
            if (page < 0 || page >= a.c.n_pages) continue;
            const int64_t row = (((int64_t)page * a.c.n_kv_heads + hk) << a.page_shift) + (j & (a.c.page_size - 1));
            const uint8_t *kc = static_cast<const uint8_t *>(a.c.k_codes) + row * (D / 2) + lane * (P / 2);
            const uint8_t *vc = static_cast<const uint8_t *>(a.c.v_codes) + row * (D / 2) + lane * (P / 2);
            const int64_t sc = row * (D / 32) + lane * P / 32;
            const float ks = __half2float(static_cast<const __half *>(a.c.k_scales)[sc]);
            const float vs = __half2float(static_cast<const __half *>(a.c.v_scales)[sc]);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) s += q[i] * (float)((int)(kc[i / 2] >> (4 * (i & 1)) & 15) - 8);
            s *= ks;
#pragma unroll
            for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
            const float mn = fmaxf(m, s);
            const float f = exp2f(m - mn), e = exp2f(s - mn);
            l = l * f + e;
#pragma unroll
            for (int i = 0; i < P; ++i)
                o[i] = o[i] * f + e * vs * (float)((int)(vc[i / 2] >> (4 * (i & 1)) & 15) - 8);
            m = mn;
        }
        const float r = l > 0.f ? rsqrt_dim<D>() / l : 0.f;
        fwht_warp<D>(o, lane);
#pragma unroll
        for (int i = 0; i < P; ++i)
            a.out[t * a.d.out_token_stride + (int64_t)h * D + lane * P + i] = __float2bfloat16_rn(o[i] * r);
    }
}

}  // namespace

extern "C" size_t strata_kv4_attention_workspace_bytes(const strata_kv4_cache *cache, int32_t n_q_heads) {
    if (strata_check_kv4_cache(cache) != STRATA_OK) return 0;
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads) return 0;
    return 16;
}

extern "C" strata_status strata_kv4_attention(const strata_kv4_cache *cache, const strata_kv4_attn_desc *d,
                                              strata_rope rope, const int32_t *positions, const void *q,
                                              const int32_t *q_offsets, const int32_t *kv_lens,
                                              const int32_t *block_table, void *out, void *workspace,
                                              size_t workspace_bytes, strata_stream_t stream) {
    const strata_status s = strata_check_kv4_cache(cache);
    if (s != STRATA_OK) return s;
    if (!d) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL desc");
    if (d->n_q_heads < 1 || d->n_q_heads % cache->n_kv_heads)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "n_q_heads %d is not a multiple of n_kv_heads %d", d->n_q_heads,
                                cache->n_kv_heads);
    if (d->n_seqs < 0 || d->n_tokens < 0 || d->max_q_len < 0 || d->max_pages < 0 || d->window < 0)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "a negative count in the desc");
    if (!std::isfinite(d->scale)) return strata_set_error(STRATA_ERR_INVALID_ARG, "scale is not finite");
    if ((int64_t)d->max_pages * cache->page_size > 0x7fffffff || d->n_tokens > 0x7fffffff)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "2^31 positions or query rows");
    if (rope && rope->desc.head_dim != cache->head_dim)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "the rotary handle has head_dim %d, the cache %d",
                                rope->desc.head_dim, cache->head_dim);
    if (d->n_seqs == 0 || d->n_tokens == 0) return STRATA_OK;
    if (!q || !out || !q_offsets || !kv_lens || (!block_table && d->max_pages > 0) || (rope && !positions) || !workspace)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL tensor pointer");
    if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(workspace)) & 15)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "q, out and workspace must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(q_offsets) | reinterpret_cast<uintptr_t>(kv_lens) |
         reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(positions)) & 3)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    const int64_t row = (int64_t)d->n_q_heads * cache->head_dim;
    if (((d->q_token_stride | d->out_token_stride) & 7) ||
        (d->n_tokens > 1 && (d->q_token_stride < row || d->out_token_stride < row)))
        return strata_set_error(STRATA_ERR_INVALID_ARG,
                                "token strides must be multiples of 8 elements and hold the heads of a token");
    const size_t need = strata_kv4_attention_workspace_bytes(cache, d->n_q_heads);
    if (workspace_bytes < need)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "workspace of %zu bytes, %zu needed", workspace_bytes, need);
    static const RopeTable none = {};
    const RopeTable &tab = rope ? rope->table : none;
    AttnArgs a{*cache, *d, positions, static_cast<const __nv_bfloat16 *>(q), q_offsets, kv_lens, block_table,
               static_cast<__nv_bfloat16 *>(out), d->n_q_heads / cache->n_kv_heads, 0, 0.f};
    while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
    a.scale_log2 = d->scale * 1.44269504088896340736f;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int gx = d->max_q_len < 1 ? 1 : d->max_q_len < 65536 ? d->max_q_len : 65536;
    const dim3 grid(gx, (d->n_q_heads + 3) / 4, d->n_seqs);
    if (cache->head_dim == 64)
        k_attn_rows<64><<<grid, 128, 0, st>>>(tab, a);
    else if (cache->head_dim == 128)
        k_attn_rows<128><<<grid, 128, 0, st>>>(tab, a);
    else
        k_attn_rows<256><<<grid, 128, 0, st>>>(tab, a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return strata_set_error(STRATA_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return STRATA_OK;
}
