// rope.cu -- rotary positions on bf16 head rows (include/strata_attn.h).
//
// The angle of pair i at position p is p f_i. Only its fraction of a turn
// matters, so the handle keeps f_i / (2 pi) as a 64-bit fixed-point fraction
// and the kernel multiplies by p modulo 2^64: exact for any position, where a
// product in fp32 would be off by whole radians at far ones.
//
// The kernel streams every row once (2 bytes in, 2 out per value) and is bound
// by HBM. A block takes a few tokens at a time: their cosines and sines are
// computed once (fp64, rotary_dim / 2 a token, one for each thread) into shared
// memory and serve every head; those of the block's next tokens are computed while
// this one's chunks stream, and a chunk is fetched while the one before is turned.
// Measured: 8,192 tokens of 36 heads of 128 30.8 us (4.9 TB/s), 64 tokens 6.8 us a
// call, the call's own cost. Interleaved 34.9 us (one chunk in flight a thread,
// where the half layout has two), half of the head turned 37.1 us. Widths that
// fill no chunk go value by value: 20 of 128 113 us.
#include <cmath>
#include <new>

#include "abi_internal.h"
#include "kv4_row.cuh"

using namespace strata;

namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 6;  // for an SM: bytes on their way against registers (4: 31.9 us, 6: 30.8 us for 8,192 tokens of 36 heads)

struct RopeArgs {
    const __nv_bfloat16 *x;
    __nv_bfloat16 *out;
    const int32_t *positions;
    int64_t x_tok, x_head, o_tok, o_head;
    int64_t n_tokens;
    int heads, D;
    int tokens_per_block, items;  // items: of a head
    uint64_t heads_inv, items_inv;  // for quotient()
};

// x / d for 0 <= x < 2^31 as a product with inv = 2^64 / d, rounded up (0 for
// d = 1): exact, since the rounding adds less than 2^-33 to the quotient
uint64_t inverse(int d) { return d > 1 ? ~0ull / (uint64_t)d + 1 : 0; }
__device__ __forceinline__ int quotient(int x, uint64_t inv) { return inv ? (int)__umul64hi((uint64_t)(uint32_t)x, inv) : x; }

// Whole 16-byte chunks: for the half layout a chunk of first halves and its
// chunk of second halves, for the interleaved one four pairs in one chunk;
// chunks past rotary_dim are copied. Every item reads and writes only its own
// values, so out may be x.
template <bool HALF>
__global__ void __launch_bounds__(kThreads, kBlocks) k_rope_vec(const __grid_constant__ RopeTable tab, const __grid_constant__ RopeArgs a) {
    __shared__ __align__(16) float2 cs[2][kThreads];  // [token][pair], of this group of tokens and the next
    const int pairs = tab.rd / 2;
    const int rot = HALF ? tab.rd / 16 : tab.rd / 8;  // rotated items of a head
    struct Item {
        uint4 u, v;
        __nv_bfloat16 *out;
        int c, t;
    };
    const int64_t step = (int64_t)gridDim.x * a.tokens_per_block;
    const int lt = threadIdx.x / pairs, lp = threadIdx.x - lt * pairs;
    auto angles = [&](int64_t t0, int b) {
        if (lt < a.tokens_per_block && t0 + lt < a.n_tokens) cs[b][threadIdx.x] = rope_cs(tab, lp, a.positions[t0 + lt]);
    };
    int b = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * a.tokens_per_block; t0 < a.n_tokens; t0 += step, b ^= 1) {
        const int nt = (int)min((int64_t)a.tokens_per_block, a.n_tokens - t0);
        const int total = nt * a.heads * a.items;
        auto fetch = [&](Item &x, int it) {
            const int th = quotient(it, a.items_inv);
            x.c = it - th * a.items;
            x.t = quotient(th, a.heads_inv);
            const int h = th - x.t * a.heads;
            const int64_t t = t0 + x.t;
            const int e = x.c < rot ? x.c * 8 : tab.rd + (x.c - rot) * 8;
            const __nv_bfloat16 *xr = a.x + t * a.x_tok + h * a.x_head + e;
            x.out = a.out + t * a.o_tok + h * a.o_head + e;
            x.u = *reinterpret_cast<const uint4 *>(xr);
            if (HALF && x.c < rot) x.v = *reinterpret_cast<const uint4 *>(xr + pairs);
        };
        Item cur, next;
        int it = threadIdx.x;
        if (it < total) fetch(next, it);
        if (t0 == (int64_t)blockIdx.x * a.tokens_per_block) {
            angles(t0, 0);
            __syncthreads();
        }
        angles(t0 + step, b ^ 1);
        for (; it < total; it += kThreads) {
            cur = next;
            if (it + kThreads < total) fetch(next, it + kThreads);
            if (cur.c >= rot) {  // not rotated
                *reinterpret_cast<uint4 *>(cur.out) = cur.u;
                continue;
            }
            // four or eight pairs, two for each 16-byte load
            const float4 *c = reinterpret_cast<const float4 *>(cs[b] + cur.t * pairs + cur.c * (HALF ? 8 : 4));
            const uint32_t u[4] = {cur.u.x, cur.u.y, cur.u.z, cur.u.w};
            if constexpr (HALF) {
                const uint32_t v[4] = {cur.v.x, cur.v.y, cur.v.z, cur.v.w};
                uint32_t ru[4], rv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 k = c[j];
                    const float2 c0 = make_float2(k.x, k.y), c1 = make_float2(k.z, k.w);
                    ru[j] = pack_bf16(rope_first(bf16_lo(u[j]), bf16_lo(v[j]), c0),
                                      rope_first(bf16_hi(u[j]), bf16_hi(v[j]), c1));
                    rv[j] = pack_bf16(rope_second(bf16_lo(u[j]), bf16_lo(v[j]), c0),
                                      rope_second(bf16_hi(u[j]), bf16_hi(v[j]), c1));
                }
                *reinterpret_cast<uint4 *>(cur.out) = make_uint4(ru[0], ru[1], ru[2], ru[3]);
                *reinterpret_cast<uint4 *>(cur.out + pairs) = make_uint4(rv[0], rv[1], rv[2], rv[3]);
            } else {
                uint32_t r[4];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    const float4 k = c[j / 2];
                    const float2 c0 = make_float2(k.x, k.y), c1 = make_float2(k.z, k.w);
                    r[j] = pack_bf16(rope_first(bf16_lo(u[j]), bf16_hi(u[j]), c0), rope_second(bf16_lo(u[j]), bf16_hi(u[j]), c0));
                    r[j + 1] = pack_bf16(rope_first(bf16_lo(u[j + 1]), bf16_hi(u[j + 1]), c1),
                                         rope_second(bf16_lo(u[j + 1]), bf16_hi(u[j + 1]), c1));
                }
                *reinterpret_cast<uint4 *>(cur.out) = make_uint4(r[0], r[1], r[2], r[3]);
            }
        }
        __syncthreads();  // the next group's angles are there, these are done with
    }
}

// rotary_dim that does not fill whole chunks: one pair, or one value past
// rotary_dim, at a time
__global__ void __launch_bounds__(kThreads) k_rope_scalar(const __grid_constant__ RopeTable tab, RopeArgs a) {
    __shared__ float2 cs[STRATA_ROPE_MAX_HEAD_DIM / 2];
    const int pairs = tab.rd / 2;
    const int items = pairs + a.D - tab.rd;
    for (int64_t t = blockIdx.x; t < a.n_tokens; t += gridDim.x) {
        const int pos = a.positions[t];
        for (int i = threadIdx.x; i < pairs; i += kThreads) cs[i] = rope_cs(tab, i, pos);
        __syncthreads();
        for (int it = threadIdx.x; it < items * a.heads; it += kThreads) {
            const int h = it / items, c = it - h * items;
            const __nv_bfloat16 *xr = a.x + t * a.x_tok + h * a.x_head;
            __nv_bfloat16 *orow = a.out + t * a.o_tok + h * a.o_head;
            if (c >= pairs) {
                orow[tab.rd + c - pairs] = xr[tab.rd + c - pairs];
            } else {
                const int iu = tab.half ? c : 2 * c, iv = tab.half ? c + pairs : 2 * c + 1;
                const float u = __bfloat162float(xr[iu]), v = __bfloat162float(xr[iv]);
                orow[iu] = __float2bfloat16_rn(rope_first(u, v, cs[c]));
                orow[iv] = __float2bfloat16_rn(rope_second(u, v, cs[c]));
            }
        }
        __syncthreads();
    }
}

// rows one behind the other, token by token or head by head
bool rows_apart(int64_t tok, int64_t head, int64_t tokens, int64_t heads, int D) {
    auto holds = [&](int64_t inner, int64_t n_inner, int64_t outer, int64_t n_outer) {
        return (n_inner == 1 || inner >= D) && (n_outer == 1 || outer >= (__int128)(n_inner - 1) * inner + D);
    };
    return holds(head, heads, tok, tokens) || holds(tok, tokens, head, heads);
}
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

extern "C" strata_status strata_rope_create(const strata_rope_desc *d, strata_rope *out) {
    if (!d || !out) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL desc or out");
    *out = nullptr;
    if (d->layout != STRATA_ROPE_HALF && d->layout != STRATA_ROPE_INTERLEAVED)
        return strata_set_error(STRATA_ERR_UNSUPPORTED, "rotary layout %d", d->layout);
    if (d->scaling < STRATA_ROPE_SCALE_NONE || d->scaling > STRATA_ROPE_SCALE_YARN)
        return strata_set_error(STRATA_ERR_UNSUPPORTED, "rotary scaling %d", d->scaling);
    if (d->head_dim < 8 || d->head_dim > STRATA_ROPE_MAX_HEAD_DIM || d->head_dim % 8)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "head_dim %d is not a multiple of 8 in 8..256", d->head_dim);
    if (d->rotary_dim < 2 || d->rotary_dim > d->head_dim || d->rotary_dim % 2)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "rotary_dim %d is not even in 2..%d", d->rotary_dim, d->head_dim);
    if (!std::isfinite(d->theta) || !(d->theta > 1.0))
        return strata_set_error(STRATA_ERR_INVALID_ARG, "theta must be finite and above 1");
    const bool scaled = d->scaling != STRATA_ROPE_SCALE_NONE;
    if (scaled && (!std::isfinite(d->factor) || !(d->factor >= 1.0)))
        return strata_set_error(STRATA_ERR_INVALID_ARG, "factor must be finite and at least 1");
    if (!std::isfinite(d->attn_factor) || d->attn_factor < 0.0)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "attn_factor must be finite and not negative");
    if (d->scaling == STRATA_ROPE_SCALE_NTK && d->rotary_dim < 4)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "NTK scaling needs rotary_dim of at least 4");
    double fast = d->beta_fast, slow = d->beta_slow;
    if (d->scaling == STRATA_ROPE_SCALE_YARN) {
        if (d->original_max_position <= 0)
            return strata_set_error(STRATA_ERR_INVALID_ARG, "YaRN needs original_max_position above 0");
        if (fast == 0.0 && slow == 0.0) fast = 32.0, slow = 1.0;
        if (!std::isfinite(fast) || !std::isfinite(slow) || !(slow > 0.0) || !(fast > slow))
            return strata_set_error(STRATA_ERR_INVALID_ARG, "YaRN needs beta_fast > beta_slow > 0");
    }
    strata_rope_s *r = new (std::nothrow) strata_rope_s();
    if (!r) return strata_set_error(STRATA_ERR_OOM, "host memory of a rotary handle");
    r->desc = *d;
    const int n = d->rotary_dim / 2;
    const double rd = d->rotary_dim;
    double theta = d->theta;
    if (d->scaling == STRATA_ROPE_SCALE_NTK) theta *= std::pow(d->factor, rd / (rd - 2.0));
    double lo = 0, hi = 0;
    if (d->scaling == STRATA_ROPE_SCALE_YARN) {
        auto pair_of = [&](double turns) {
            return rd * std::log(d->original_max_position / (turns * 2 * M_PI)) / (2 * std::log(theta));
        };
        lo = std::fmax(std::floor(pair_of(fast)), 0.0);
        hi = std::fmin(std::ceil(pair_of(slow)), rd - 1);
    }
    for (int i = 0; i < n; ++i) {
        double f = std::pow(theta, -2.0 * i / rd);
        if (d->scaling == STRATA_ROPE_SCALE_LINEAR) f /= d->factor;
        if (d->scaling == STRATA_ROPE_SCALE_YARN) {
            const double w = hi - lo != 0.0 ? hi - lo : 0.001;
            const double ramp = std::fmin(std::fmax((i - lo) / w, 0.0), 1.0);
            f = f / d->factor * ramp + f * (1 - ramp);
        }
        // turns per position, 64 fractional bits (f <= 1: below a sixth of a turn)
        r->table.freq[i] = (uint64_t)((long double)f / (2 * 3.14159265358979323846264338327950288L) * 0x1p64L + 0.5L);
    }
    r->table.m = d->attn_factor > 0.0                          ? d->attn_factor
                 : d->scaling == STRATA_ROPE_SCALE_YARN ? 0.1 * std::log(d->factor) + 1.0
                                                        : 1.0;
    r->table.rd = d->rotary_dim;
    r->table.half = d->layout == STRATA_ROPE_HALF;
    *out = r;
    return STRATA_OK;
}

extern "C" strata_status strata_rope_destroy(strata_rope rope) {
    delete rope;
    return STRATA_OK;
}

extern "C" strata_status strata_rope_apply(strata_rope rope, const void *x, int64_t x_token_stride,
                                           int64_t x_head_stride, const int32_t *positions, int64_t n_tokens,
                                           int32_t n_heads, void *out, int64_t out_token_stride,
                                           int64_t out_head_stride, strata_stream_t stream) {
    if (!rope) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL rotary handle");
    if (n_tokens < 0 || n_heads < 0) return strata_set_error(STRATA_ERR_INVALID_ARG, "negative n_tokens or n_heads");
    if (n_tokens == 0 || n_heads == 0) return STRATA_OK;
    if (!x || !out || !positions) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!aligned16(x) || !aligned16(out) || (reinterpret_cast<uintptr_t>(positions) & 3))
        return strata_set_error(STRATA_ERR_INVALID_ARG, "x and out must be 16-byte, positions 4-byte aligned");
    if ((x_token_stride | x_head_stride | out_token_stride | out_head_stride) & 7)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
    const int D = rope->desc.head_dim;
    if (!rows_apart(x_token_stride, x_head_stride, n_tokens, n_heads, D) ||
        !rows_apart(out_token_stride, out_head_stride, n_tokens, n_heads, D))
        return strata_set_error(STRATA_ERR_INVALID_ARG,
                                "strides must keep rows of head_dim values apart, token by token or head by head");
    if (n_heads > (1 << 20)) return strata_set_error(STRATA_ERR_INVALID_ARG, "n_heads %d", n_heads);
    RopeArgs a{static_cast<const __nv_bfloat16 *>(x), static_cast<__nv_bfloat16 *>(out), positions,
               x_token_stride, x_head_stride, out_token_stride, out_head_stride, n_tokens, n_heads, D, 1, 0, 0, 0};
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const RopeTable &tab = rope->table;
    if (tab.rd % (tab.half ? 16 : 8) == 0) {
        // as many tokens as threads have pairs to compute, but blocks for every SM first
        a.items = (tab.half ? tab.rd / 16 : tab.rd / 8) + (D - tab.rd) / 8;
        const int64_t fit = ((int64_t)1 << 26) / ((int64_t)n_heads * a.items);  // 32-bit indices
        int64_t most = kThreads / (tab.rd / 2);
        most = most < fit ? most : fit;
        const int64_t spread = (n_tokens + kBlocks * 148 - 1) / (kBlocks * 148);
        a.tokens_per_block = (int)(most < spread ? most : spread);
        a.heads_inv = inverse(n_heads);
        a.items_inv = inverse(a.items);
        const int64_t blocks = (n_tokens + a.tokens_per_block - 1) / a.tokens_per_block;
        const int grid = (int)(blocks < kBlocks * 148 ? blocks : kBlocks * 148);
        if (tab.half)
            k_rope_vec<true><<<grid, kThreads, 0, st>>>(tab, a);
        else
            k_rope_vec<false><<<grid, kThreads, 0, st>>>(tab, a);
    } else {
        k_rope_scalar<<<(int)(n_tokens < 65536 ? n_tokens : 65536), kThreads, 0, st>>>(tab, a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return strata_set_error(STRATA_ERR_CUDA, "rotary launch: %s", cudaGetErrorString(e));
    return STRATA_OK;
}
