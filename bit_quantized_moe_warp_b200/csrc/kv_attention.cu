// kv_attention.cu -- attention over the paged 4-bit KV cache
// (include/strata_attn.h).
//
// H is symmetric and orthonormal up to sqrt(D), so q . k' = (H q / sqrt D) . y
// for the stored row y = (c - 8) s, and sum_j p_j v'_j = H (sum_j p_j y_j) / sqrt D:
// a query row is rotated once on the way in and its output once on the way
// out, and the cache's rows are used as they are stored.
#include <cmath>

#include "abi_internal.h"
#include "kv_attn.cuh"

using namespace strata;

namespace {


// ---------------------------------------------------------------- few rows
// k_attn_split: up to 8 NT query rows of a KV head (tokens x heads of the
// group) against a long cache, which is read once. Floor: HBM, 36 D bytes a
// 32-key tile; a tile takes about 740 warp instructions, so everything around
// the matrix instructions is counted.
//
//   * S^T = K Q^T: keys are the 16 rows of m16n8k16, 8 query rows its columns.
//     A code's nibble under the exponent of 1024 (or, at bits 4..7, of 64) is
//     the exact fp16 value 1024 + c (64 + c). A block's sum is scaled in fp32,
//     so keys are never rounded; the offsets' share, -sum_b s_b sum_i q_i
//     (offset + 8), is one product more, of the scales with the query's block
//     sums (fp16 in two parts).
//   * O^T = V^T P^T: nibbles of two keys side by side, c - 8 exact in fp16;
//     the probability takes the value's scale, p s, in fp16. Weights are
//     2^(x - M + 6), so that a long tail under one large weight stays among
//     fp16's normal numbers. Where a tile's scales are not all below 2^4 with
//     some above 2^-6, a key enters with its own exponent e of them: 2^(x + e -
//     M + 6) times s 2^(1 - e) in [2, 4), and the sum l takes the weight by 2^-e.
//   * M moves only when a weight would pass 2^11: most tiles need no reduction
//     over lanes.
//
// Work: the tiles of all (sequence, KV head, row group) in a row, cut into
// equal runs of units, one for each CTA (one tile for each of the 8 warps), so that
// any mix of lengths fills the machine. A run that covers a sequence's whole
// cache writes its rows; the others leave (M, l, O) in the workspace, two at
// most for a CTA, and k_attn_join adds them up in a fixed order.
//
// Measured (B200, with the join, calls back to back): 1 token of 32 heads at
// 131,072 cached tokens of 4 KV heads of 128 30.8 us (2.4 TB/s of the cache's
// 75.5 MB), 64 sequences of 1,024 to 16,384 69 us (3.3 TB/s), 1 at 777 11 us.
// About 10 us of each are fixed: three dependent loads (lengths, page table,
// tile) before the first product, the join of the warps and of the CTAs. Over
// the whole kernel ncu shows 2.3 of 4 instructions issued a cycle and SM with 16
// warps on it: neither issue nor HBM (2.8 TB/s) is full, the rest is latency. Of
// the 740 instructions for 32 keys 245 unpack and add up values.
// 12 warps instead of 8 for 16 rows: no faster (51 and 54 us, 32 rows, 100,000
// keys); 2 blocks of 128 registers for 16 rows of 64 values: the same.
constexpr int kSplitParts = 2 * 16 * kSms;  // rows of partial results: 2 x 8 rows x 296 CTAs or 2 x 16 x 148
constexpr int kSplitWarps = 8;
// Rows of a KV head and sequence up to which k_attn_split is launched, 16 at a
// time (8 for head_dim 256), and above which k_attn_tiles. us with one and the
// other, 4 KV heads:
//   rows                     8 of 2,048 to 32,768   4 of 500 to 2,000   1 of 100,000
//   head_dim 64    32               53  69               13  17            35  46
//                  48               72  72               14  18            47  48
//                  64               94  72               15  19            59  50
//   head_dim 128   32               72 123               15  21            49  68
//                  48              101 127               17  23            67  68
//                  64              131 129               19  24            84  70
//   head_dim 256   32              155 176               20  26           104 126
//                  48              225 180               23  29           148 130
//                  64              294 181               28  30           193 131
// Set where long contexts of 64 and 128 change sides; those of 256 would before,
// short ones of any size later. Both kernels take any number.
constexpr int kSplitMostRows = 48;
constexpr int kStages = 2;  // a warp's own work on a tile covers the latency of the next
constexpr int kTile = 32;   // keys, as two halves of 16: no half crosses a page

template <int D, int NT>
struct Split {
    static constexpr int NB = D / 32;
    static constexpr int ROWS = 8 * NT;
    static constexpr int STAGE = 36 * D;             // codes 32 D, scales 4 D
    static constexpr int RING = kStages * STAGE;     // of a warp; holds its rows of O at a piece's end
    static constexpr int OROW = D + 4;
    static constexpr int SCRATCH = 2 * D + 32 * 8;   // scaled V scales of a tile, (e, 2^-e) of its keys
    static constexpr int PART = D + 4;               // floats of a part in the workspace: O, M, l
    static constexpr int SMEM = kSplitWarps * (RING + SCRATCH) + ROWS * D * 2 + ROWS * NB * 4 * 2 + ROWS * 4 +
                                2 * kSplitWarps * ROWS * 4 + 128;
    static_assert(ROWS * OROW * 4 <= RING, "O of a warp fits its ring");
    static constexpr int CTAS_PER_SM = NT == 1 && D <= 128 ? 2 : 1;
    static constexpr int CTAS = kSms * CTAS_PER_SM;
    static_assert(2 * ROWS * CTAS <= kSplitParts && CTAS <= kSplitMaxCtas, "workspace");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// (w & mask) | bits in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
__device__ __forceinline__ __half2 bits_h2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }

template <int OFF = 0>
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(v) : "r"(addr), "n"(OFF) : "memory");
    return v;
}
template <int W>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[W]) {
    if constexpr (W == 1) asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr) : "memory");
    if constexpr (W == 2) asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr) : "memory");
    if constexpr (W >= 4)
#pragma unroll
        for (int i = 0; i < W; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(addr + 4 * i) : "memory");
}
__device__ __forceinline__ uint32_t lds_half(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// 16-byte chunk c of row r of a code tile: shifted so that both readers, 8
// rows at one chunk and every second row at one chunk, meet 32 banks
template <int D>
__device__ __forceinline__ int code_chunk(int r, int c) {
    constexpr int NB = D / 32;
    const int x = D == 64 ? (r >> 2) & 1 : D == 128 ? (r >> 1) & 3 : r & 7;
    return r * (D / 2) + ((c ^ x) & (NB - 1)) * 16;
}
// Within 16-key tiles x(r + 8) = x(r), and for even r x(r + 1) = x(r) (^ 1 for
// D = 256): a lane needs one address, one XOR for each block.

struct Seq : SeqBase {
    int tile0, tiles, groups;
};
__device__ __forceinline__ Seq seq_of(const AttnArgs &a, int b, int rows_per_group) {
    Seq s;
    load_seq(s, a, b);
    const int64_t first = a.d.window > 0 ? max((int64_t)0, (int64_t)s.L - s.n - a.d.window + 1) : 0;
    s.tile0 = (int)(min(first, (int64_t)s.L) / kTile);
    s.tiles = (int)(((int64_t)s.L + kTile - 1) / kTile) - s.tile0;
    s.groups = (int)(((int64_t)s.n * a.group + rows_per_group - 1) / rows_per_group);
    return s;
}
// units of one (KV head, row group): those that stand for what a piece of it
// costs besides its tiles (rows in, warps joined, results out), then its tiles;
// one at least, which writes the zeros of a sequence without keys
// us with 0, 1, 2, 4 (head_dim 128): 64 sequences up to 16,384 74.5, 70.1, 69.4, 74.0; 8 of 6
// tokens up to 32,768 58.6, 55.1, 53.6, 53.3; 64 up to 1,500 23, 20, 20, 21.7.
constexpr int kSplitHead = 2;
__device__ __forceinline__ int seq_units(const Seq &s) { return kSplitHead + max((s.tiles + kSplitWarps - 1) / kSplitWarps, 1); }

template <int D, int NT>
__global__ void __launch_bounds__(kSplitWarps * 32, (Split<D, NT>::CTAS_PER_SM))
    k_attn_split(const __grid_constant__ RopeTable tab, const __grid_constant__ AttnArgs a) {
    using C = Split<D, NT>;
    constexpr int NB = C::NB, ROWS = C::ROWS, P = D / 32;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    uint8_t *ring = smem + warp * C::RING;
    uint8_t *scratch = smem + kSplitWarps * C::RING + warp * C::SCRATCH;
    __half *sq = reinterpret_cast<__half *>(smem + kSplitWarps * (C::RING + C::SCRATCH));
    __half *scorr = sq + ROWS * D;  // [ROWS][2][NB]: the two parts of a block's offset sum
    float *sfac = reinterpret_cast<float *>(scorr + ROWS * NB * 4);
    float *sM = sfac + ROWS, *sl = sM + kSplitWarps * ROWS;
    __shared__ int64_t s_sum[kSplitWarps];
    __shared__ int64_t s_before;
    __shared__ int s_b;
    griddep_launch_dependents();
    griddep_wait();

    // ---- this CTA's run of units, and the sequence it starts in
    int64_t total = 0, u_lo = 0, u_hi = 0, run = 0, inc = 0, v = 0;
    int ctas = 0;
    constexpr int kChunk = kSplitWarps * 32;
    auto scan = [&](int b0) {  // inc: units up to and with sequence b0 + threadIdx.x; run: with the whole chunk
        const int b = b0 + threadIdx.x;
        v = 0;
        if (b < a.d.n_seqs) {
            const Seq s = seq_of(a, b, ROWS);
            v = (int64_t)seq_units(s) * s.groups * a.c.n_kv_heads;
        }
        inc = v;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(kFullMask, inc, x);
            if (lane >= x) inc += o;
        }
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        inc += run;
#pragma unroll
        for (int w = 0; w < kSplitWarps; ++w) {
            const int64_t o = s_sum[w];
            if (w < warp) inc += o;
            run += o;
        }
        __syncthreads();
    };
    // Up to 64 sequences: every warp for itself, two for each lane
    const bool few = a.d.n_seqs <= 64;
    Seq mine[2] = {};
    if (few) {
        int64_t w[2], upto = 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            w[k] = 0;
            if (2 * lane + k < a.d.n_seqs) {
                mine[k] = seq_of(a, 2 * lane + k, ROWS);
                w[k] = (int64_t)seq_units(mine[k]) * mine[k].groups * a.c.n_kv_heads;
            }
        }
        upto = w[0] + w[1];
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(kFullMask, upto, x);
            if (lane >= x) upto += o;
        }
        run = __shfl_sync(kFullMask, upto, 31);
        inc = upto, v = w[0] + w[1];
    } else {
        for (int b0 = 0; b0 < a.d.n_seqs; b0 += kChunk) scan(b0);
    }
    total = run;
    ctas = (int)min(total, (int64_t)C::CTAS);  // a unit each at least
    Seq s{};
    int b = 0;
    int64_t before = 0;
    if (blockIdx.x < ctas) {
        u_lo = run_start(total, blockIdx.x, ctas);
        u_hi = run_start(total, blockIdx.x + 1, ctas);
        if (few) {
            const int src = __ffs(__ballot_sync(kFullMask, u_lo < inc)) - 1;
            const int64_t w0 = (int64_t)seq_units(mine[0]) * mine[0].groups * a.c.n_kv_heads;
            const bool second = 2 * lane + 1 < a.d.n_seqs && inc - v + w0 <= u_lo;
            const Seq t = second ? mine[1] : mine[0];
            b = 2 * src + (__shfl_sync(kFullMask, second ? 1 : 0, src));
            before = __shfl_sync(kFullMask, second ? inc - v + w0 : inc - v, src);
            s.t0 = __shfl_sync(kFullMask, t.t0, src);
            s.n = __shfl_sync(kFullMask, t.n, src), s.L = __shfl_sync(kFullMask, t.L, src);
            s.tile0 = __shfl_sync(kFullMask, t.tile0, src), s.tiles = __shfl_sync(kFullMask, t.tiles, src);
            s.groups = __shfl_sync(kFullMask, t.groups, src);
        } else {
            int b0 = 0;
            if (a.d.n_seqs > kChunk) {
                run = 0;
                for (b0 = -kChunk; run <= u_lo;) scan(b0 += kChunk);
            }
            if (inc - v <= u_lo && u_lo < inc) {
                s_b = b0 + threadIdx.x;
                s_before = inc - v;
            }
            __syncthreads();
            b = uniform(s_b);
            before = s_before;
            s = seq_of(a, b, ROWS);
        }
    }
    Span *spans = static_cast<Span *>(a.workspace);
    float *parts = reinterpret_cast<float *>(spans + kSplitMaxCtas);
    if (threadIdx.x == 0) spans[blockIdx.x].parts = 0;
    if (u_lo == u_hi) return;
    auto settle = [&]() {
        s.n = uniform(s.n), s.L = uniform(s.L), s.tile0 = uniform(s.tile0), s.tiles = uniform(s.tiles);
        s.groups = uniform(s.groups);
    };
    settle();
    // from here on units count from u_lo
    int per = seq_units(s);
    int vh = uniform((int)run_start(u_lo - before, 1, per));  // (KV head, row group) inside the sequence
    int first = uniform((int)(before + (int64_t)vh * per - u_lo));  // its first unit
    const int units = uniform((int)(u_hi - u_lo));
    const uint32_t n_pages = (uint32_t)min(a.c.n_pages, (int64_t)0x80000000);
    const uint32_t ring_u = smem_u32(ring), scratch_u = smem_u32(scratch);
    const uint32_t lane_chunk = code_chunk<D>(lane / NB, lane % NB);

    int count = 0;  // pieces
    for (int u = 0; u < units;) {
        const int u_end = min(first + per, units);
        const int t_lo = max(u - first - kSplitHead, 0), t_hi = u_end - first - kSplitHead;
        if (t_hi <= t_lo) break;  // the run ends before the first tile
        const int rg = vh / a.c.n_kv_heads, hk = vh - rg * a.c.n_kv_heads;
        const int row0 = rg * ROWS;
        const int rows = min(ROWS, s.n * a.group - row0);
        const int p_first = s.L - s.n;           // position of query 0

        // ---- the warp's tiles: tile0 + 8 unit + warp
        int it = s.tile0 + t_lo * kSplitWarps + warp;
        const int t_end = min(s.tile0 + s.tiles, s.tile0 + t_hi * kSplitWarps);
        const int32_t *table = a.table + (int64_t)b * a.d.max_pages;
        int nit = it;                            // next tile to ask for
        uint32_t page[2] = {~0u, ~0u}, there = 0;  // the pages of its halves; bit 2 s + h: half h of stage s is there
        auto pages = [&]() {
            if (nit < t_end) {
                page[0] = __ldg(table + (nit * kTile >> a.page_shift));
                page[1] = nit * kTile + 16 < s.L ? __ldg(table + ((nit * kTile + 16) >> a.page_shift)) : ~0u;
            } else {
                page[0] = page[1] = ~0u;
            }
        };
        pages();
        auto issue = [&](int stage) {
            const uint32_t st = ring_u + stage * C::STAGE;
            there &= ~(3u << 2 * stage);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t pg = uniform(page[h]);
                if (pg < n_pages) {
                    there |= 1u << (2 * stage + h);
                    const uint32_t row = ((pg * a.c.n_kv_heads + hk) << a.page_shift) +
                                         ((nit * kTile + 16 * h) & (a.c.page_size - 1));
                    const uint8_t *kc = static_cast<const uint8_t *>(a.c.k_codes) + (uint64_t)row * (D / 2) + lane * 16;
                    const uint8_t *vc = static_cast<const uint8_t *>(a.c.v_codes) + (uint64_t)row * (D / 2) + lane * 16;
#pragma unroll
                    for (int i = 0; i < (16 * NB + 31) / 32; ++i) {
                        // lanes 32 chunks on lie 32 / NB rows on: the shift is the same for D = 64 and 128
                        const uint32_t to = st + h * 8 * D + (D == 256 ? code_chunk<D>(lane / NB + i * (32 / NB), lane % NB)
                                                                       : lane_chunk + i * 512);
                        cp_async16(to, kc + i * 512);
                        cp_async16(to + 16 * D, vc + i * 512);
                    }
                    if (lane < 4 * NB) {         // scales: 2 NB chunks of keys, then of values
                        const bool v = lane >= 2 * NB;
                        const uint8_t *sc = static_cast<const uint8_t *>(v ? a.c.v_scales : a.c.k_scales) + lane * 16;
                        // D bytes a half: 2 NB chunks of 16
                        cp_async16(st + 32 * D + h * D + (v ? D : 0) + lane * 16, sc - (v ? D : 0) + (uint64_t)row * (D / 16));
                    }
                }
            }
            cp_async_commit();
            nit += kSplitWarps;
            pages();
        };
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(i);

        // ---- query rows: rotary, transform, fp16 with a power-of-two scale
        for (int r = warp; r < ROWS; r += kSplitWarps) {
            float v[P];
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = 0.f;
            if (r < rows) {
                const int i = by_group(a, row0 + r), h = hk * a.group + (row0 + r) - i * a.group;
                const int64_t tok = s.t0 + i;
                typename QueryRow<D>::Raw raw;
                float2 cs[P];
                QueryRow<D>::load(raw, a.q + tok * a.d.q_token_stride + (int64_t)h * D, tab, lane);
                QueryRow<D>::angles(cs, tab, tab.rd ? a.positions[tok] : 0, lane);
                QueryRow<D>::turn(v, raw, cs, tab, 1.f, lane);
            }
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
            for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, x));
            const uint32_t ex = min(max(__float_as_uint(m) >> 23, 1u), 252u);
            const float mul = m > 0.f ? __uint_as_float((253u - ex) << 23) : 1.f;  // largest value to [0.5, 1)
            float corr = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int d = lane * P + i, n = d & 7;
                const __half q = __float2half_rn(v[i] * mul);
                sq[r * D + (d & ~7) + (n < 4 ? 2 * n : 2 * n - 7)] = q;
                corr = fmaf(__half2float(q), (d & 1) ? -72.f : -1032.f, corr);
            }
#pragma unroll
            for (int x = 1; x < 32 / NB; x <<= 1) corr += __shfl_xor_sync(kFullMask, corr, x);
            if ((lane & (32 / NB - 1)) == 0) {  // at most 1032 * 32 in magnitude
                const __half c0 = __float2half_rn(corr);
                scorr[r * 2 * NB + lane / (32 / NB)] = c0;
                scorr[r * 2 * NB + NB + lane / (32 / NB)] = __float2half_rn(corr - __half2float(c0));
            }
            if (lane == 0) sfac[r] = a.scale_log2 * (m > 0.f ? __uint_as_float((ex + 1) << 23) : 1.f);
        }
        __syncthreads();
        uint32_t qf[NT][NB][4];
        uint32_t cf[NT][2];
        float fac[NT][2], M[NT][2], l[NT][2], o[NT][2 * NB][4];
        int hi[NT][2], lo[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint4 w = *reinterpret_cast<const uint4 *>(sq + (n * 8 + g) * D + 32 * k + 8 * t);
                qf[n][k][0] = w.x, qf[n][k][1] = w.y, qf[n][k][2] = w.z, qf[n][k][3] = w.w;
            }
            // row n * 8 + g: offset sums of blocks 2t, 2t + 1 against the scales (D < 256: both parts in one half of k)
            const uint32_t *sc = reinterpret_cast<const uint32_t *>(scorr + (n * 8 + g) * 2 * NB);
            cf[n][0] = t < NB ? sc[t] : 0u;
            cf[n][1] = NB == 8 ? sc[t + 4] : 0u;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = n * 8 + 2 * t + j;
                fac[n][j] = sfac[r];
                const int p = p_first + by_group(a, row0 + r);
                hi[n][j] = min(p, s.L - 1);
                lo[n][j] = a.d.window > 0 ? (int)max((int64_t)p - a.d.window, (int64_t)-1) : -1;
                M[n][j] = -FLT_MAX;
                l[n][j] = 0.f;
            }
#pragma unroll
            for (int k = 0; k < 2 * NB; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[n][k][j] = 0.f;
        }
        // tiles up to here, and from there on, need no mask
        const int last_row = by_group(a, row0 + rows - 1);
        const int full_hi = p_first + by_group(a, row0);
        const int full_lo = a.d.window > 0 ? (int)max((int64_t)p_first + last_row - a.d.window, (int64_t)-1) : -1;
        // keys that no row sees, (.., any_lo] and [any_hi, ..), may hold anything
        const int any_lo = a.d.window > 0 ? (int)max((int64_t)full_hi - a.d.window, (int64_t)-1) : -1;
        const int any_hi = min(p_first + last_row + 1, s.L);

        // word t of block 0 of key g; word g / 2 of block 0 of key 2t, and the half of it with values 4g .. 4g + 3
        const uint32_t k_base = code_chunk<D>(g, 0) + 4 * t, v_base = 16 * D + code_chunk<D>(2 * t, 0) + 4 * (g >> 1);
        const uint32_t sel = (g & 1) ? 0x7632u : 0x5410u;  // values 4g .. 4g + 3 of a block
        float *ve = reinterpret_cast<float *>(scratch + 2 * D);       // [32 keys] (e, 2^-e)
        const float zero[4] = {0.f, 0.f, 0.f, 0.f};
        for (int stage = 0; it < t_end; it += kSplitWarps, stage ^= 1) {
            cp_async_wait<0>();
            __syncwarp();
            issue(stage ^ 1);
            const uint32_t have = there >> 2 * stage & 3;
            if (!have) continue;
            const uint32_t st = ring_u + stage * C::STAGE;
            const int j0 = it * kTile;
            const bool full = have == 3 && j0 + kTile - 1 < any_hi && j0 > any_lo;

            // V scales in key pairs, [2][8 pairs][NB] half2
            float2 e[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) e[h][0] = e[h][1] = make_float2(0.f, 1.f);
            {
                constexpr int N = (NB + 3) / 4;
                uint32_t x[2][N], m = 0;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint32_t at = st + 34 * D + h * D + (2 * g * NB + ((t + 4 * i) & (NB - 1))) * 2;
                        x[h][i] = lds_half(at) | lds_half(at + 2 * NB) << 16;
                    }
                if (!full) {  // whatever no row sees or was never copied
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = j0 + 16 * h + 2 * g;
                        const uint32_t keep = have >> h & 1 ? (j < any_hi && j > any_lo ? 0xffffu : 0u) |
                                                                  (j + 1 < any_hi && j >= any_lo ? 0xffff0000u : 0u)
                                                            : 0u;
#pragma unroll
                        for (int i = 0; i < N; ++i) x[h][i] &= keep;
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < N; ++i) m = max(max(m, x[h][i] << 17), (x[h][i] & 0x7fff0000u) << 1);
                const bool large = m >= 0x4c00u << 17, fair = m >= 0x2400u << 17;
                const uint32_t to = scratch_u + (g * NB + t) * 4;
                if (!__any_sync(kFullMask, large) && __any_sync(kFullMask, fair)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (t + 4 * i < NB) sts32(to + h * D + 16 * i, x[h][i]);
                    __syncwarp();
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        __half2 y = __habs2(bits_h2(x[h][0]));
#pragma unroll
                        for (int i = 1; i < N; ++i) y = __hmax2(y, __habs2(bits_h2(x[h][i])));
                        y = __hmax2(y, bits_h2(__shfl_xor_sync(kFullMask, h2_bits(y), 1)));
                        y = __hmax2(y, bits_h2(__shfl_xor_sync(kFullMask, h2_bits(y), 2)));
                        const uint32_t z = __vmaxu2(h2_bits(y) & 0x7c007c00u, 0x04000400u);
                        const __half2 mul = bits_h2(0x7c007c00u - z);  // 2^(1 - exponent)
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (t + 4 * i < NB) sts32(to + h * D + 16 * i, h2_bits(__hmul2(bits_h2(x[h][i]), mul)));
                        if (t == 0) {
                            const int f0 = (int)(z >> 10 & 31) - 16, f1 = (int)(z >> 26) - 16;  // s 2^-f in [2, 4)
                            *reinterpret_cast<float4 *>(ve + 32 * h + 4 * g) =
                                make_float4((float)f0, __int_as_float((127 - f0) << 23), (float)f1,
                                            __int_as_float((127 - f1) << 23));
                        }
                    }
                    __syncwarp();
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int r = 0; r < 2; ++r) e[h][r] = *reinterpret_cast<float2 *>(ve + 32 * h + 2 * g + 16 * r);
                }
            }
            // S^T
            float x[NT][2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float ks[2][NB];
                const uint32_t sc = st + 32 * D + h * D + g * NB * 2;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    uint32_t w[NB / 2];
                    lds_words(sc + r * 16 * NB, w);
#pragma unroll
                    for (int k = 0; k < NB / 2; ++k) {
                        const float2 f = __half22float2(bits_h2(w[k]));
                        ks[r][2 * k] = f.x, ks[r][2 * k + 1] = f.y;
                    }
                }
                const uint32_t s0 = lds32(sc + (2 * t & (NB - 1)) * 2), s1 = lds32<16 * NB>(sc + (2 * t & (NB - 1)) * 2);
                const uint32_t as[4] = {s0, s1, NB == 8 ? s0 : 0u, NB == 8 ? s1 : 0u};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma16816(x[n][h], as, cf[n][0], cf[n][1], zero);
                const uint32_t base = st + k_base + h * 8 * D;
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    const uint32_t w0 = lds32(base ^ (16 * k)), w1 = lds32<4 * D>(base ^ (16 * k));
                    const uint32_t a0[4] = {and_or(w0, 0x000f000fu, 0x64006400u), and_or(w1, 0x000f000fu, 0x64006400u),
                                            and_or(w0, 0x00f000f0u, 0x54005400u), and_or(w1, 0x00f000f0u, 0x54005400u)};
                    const uint32_t h0 = w0 >> 8, h1 = w1 >> 8;
                    const uint32_t a1[4] = {and_or(h0, 0x000f000fu, 0x64006400u), and_or(h1, 0x000f000fu, 0x64006400u),
                                            and_or(h0, 0x00f000f0u, 0x54005400u), and_or(h1, 0x00f000f0u, 0x54005400u)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c[4];
                        mma16816(c, a0, qf[n][k][0], qf[n][k][1], zero);
                        mma16816(c, a1, qf[n][k][2], qf[n][k][3], c);
#pragma unroll
                        for (int j = 0; j < 4; ++j) x[n][h][j] = fmaf(c[j], ks[j >> 1][k], x[n][h][j]);
                    }
                }
            }
            // softmax: weights of keys g, g + 8 of each half for query rows 2t, 2t + 1
            const bool whole = full && j0 + kTile - 1 <= full_hi && j0 > full_lo;
            bool grow = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[n][h][j] = fmaf(x[n][h][j], fac[n][j & 1], e[h][j >> 1].x);
                if (!whole) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int pos = j0 + 16 * h + g + (j < 2 ? 0 : 8);
                            if (pos > hi[n][j & 1] || pos <= lo[n][j & 1] || !(have >> h & 1)) x[n][h][j] = -INFINITY;
                        }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    grow |= fmaxf(fmaxf(x[n][0][j], x[n][0][j + 2]), fmaxf(x[n][1][j], x[n][1][j + 2])) > M[n][j] + 11.f;
            }
            if (__any_sync(kFullMask, grow)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float m = fmaxf(fmaxf(x[n][0][j], x[n][0][j + 2]), fmaxf(x[n][1][j], x[n][1][j + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(kFullMask, m, d));
                        m = fmaxf(M[n][j], m - 6.f);
                        const float f = ex2(M[n][j] - m);
                        M[n][j] = m;
                        l[n][j] *= f;
#pragma unroll
                        for (int k = 0; k < 2 * NB; ++k) o[n][k][j] *= f, o[n][k][j + 2] *= f;
                    }
            }
            uint32_t pr[NT][2][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        x[n][h][j] = ex2(x[n][h][j] - M[n][j & 1]);
                        l[n][j & 1] = fmaf(x[n][h][j], e[h][j >> 1].y, l[n][j & 1]);
                    }
                    pr[n][h][0] = transpose8x8(h2_bits(__floats2half2_rn(x[n][h][0], x[n][h][1])));  // keys 2t, 2t + 1
                    pr[n][h][1] = transpose8x8(h2_bits(__floats2half2_rn(x[n][h][2], x[n][h][3])));  // keys 2t + 8, 2t + 9
                }
            // O^T
            const __half2 off = __floats2half2_rn(-1032.f, -1032.f), off64 = __floats2half2_rn(-72.f, -72.f);
            auto unpack = [&](uint32_t w, uint32_t (&v)[4]) {
                const uint32_t u = w >> 8;
                v[0] = h2_bits(__hadd2(bits_h2(and_or(w, 0x000f000fu, 0x64006400u)), off));
                v[1] = h2_bits(__hadd2(bits_h2(and_or(w, 0x00f000f0u, 0x54005400u)), off64));
                v[2] = h2_bits(__hadd2(bits_h2(and_or(u, 0x000f000fu, 0x64006400u)), off));
                v[3] = h2_bits(__hadd2(bits_h2(and_or(u, 0x00f000f0u, 0x54005400u)), off64));
            };
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t vs0[NB], vs1[NB];
                lds_words(scratch_u + h * D + t * NB * 4, vs0);
                lds_words(scratch_u + h * D + (t + 4) * NB * 4, vs1);
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    // keys 2t, 2t + 1 and 8 on
                    const uint32_t at = (st + v_base + h * 8 * D) ^ (16 * k), at1 = (D == 256 ? at ^ 16 : at) + D / 2;
                    const uint32_t w[4] = {lds32(at), lds32(at1), lds32<4 * D>(at), lds32<4 * D>(at1)};
                    uint32_t v0[4], v1[4];
                    unpack(__byte_perm(w[0], w[1], sel), v0);
                    unpack(__byte_perm(w[2], w[3], sel), v1);
                    const uint32_t a0[4] = {v0[0], v0[1], v1[0], v1[1]}, a1[4] = {v0[2], v0[3], v1[2], v1[3]};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const uint32_t b0 = h2_bits(__hmul2(bits_h2(pr[n][h][0]), bits_h2(vs0[k]))),
                                       b1 = h2_bits(__hmul2(bits_h2(pr[n][h][1]), bits_h2(vs1[k])));
                        mma16816(o[n][2 * k], a0, b0, b1, o[n][2 * k]);
                        mma16816(o[n][2 * k + 1], a1, b0, b1, o[n][2 * k + 1]);
                    }
                }
            }
            __syncwarp();  // the scratch is written again
        }
        cp_async_wait<0>();
        __syncwarp();

        // ---- join the 8 warps
        float *so = reinterpret_cast<float *>(ring);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = n * 8 + 2 * t + j;
                float sum = l[n][j];
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
                if (g == 0) {
                    sM[warp * ROWS + r] = M[n][j];
                    sl[warp * ROWS + r] = sum;
                }
#pragma unroll
                for (int k = 0; k < NB; ++k)
                    *reinterpret_cast<float4 *>(so + r * C::OROW + 32 * k + 4 * g) =
                        make_float4(o[n][2 * k][j], o[n][2 * k][j + 2], o[n][2 * k + 1][j], o[n][2 * k + 1][j + 2]);
            }
        __syncthreads();
        const bool whole = t_lo == 0 && u_end == first + per;
        const int slot = count ? 1 : 0;  // the first piece may go on from the CTA before, the last one into the next
        for (int r = warp; r < rows; r += kSplitWarps) {
            float m = sM[r];
#pragma unroll
            for (int w = 1; w < kSplitWarps; ++w) m = fmaxf(m, sM[w * ROWS + r]);
            float sum = 0.f, v[P];
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = 0.f;
#pragma unroll
            for (int w = 0; w < kSplitWarps; ++w) {
                const float f = ex2(sM[w * ROWS + r] - m);
                sum = fmaf(sl[w * ROWS + r], f, sum);
                const float *ow = reinterpret_cast<const float *>(smem + w * C::RING) + r * C::OROW + lane * P;
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = fmaf(ow[i], f, v[i]);
            }
            if (whole) {
                store_row<D>(a, v, sum, s.t0, hk, row0 + r, lane);
            } else {
                float *part = parts + (int64_t)((blockIdx.x * 2 + slot) * ROWS + r) * C::PART;
#pragma unroll
                for (int i = 0; i < P; ++i) part[lane * P + i] = v[i];
                if (lane == 0) part[D] = m, part[D + 1] = sum;
            }
        }
        if (t_lo == 0 && !whole && threadIdx.x == 0) {
            // it starts here and ends in the CTA that holds its last unit
            const int64_t last = u_lo + first + per - 1;
            int c = (int)run_start(ctas, last, total);  // run c starts at `last` or before it
            while (run_start(total, c + 1, ctas) <= last) ++c;
            spans[blockIdx.x] = Span{c - (int)blockIdx.x + 1, slot, (int)s.t0, rows, hk, row0, {0, 0}};
        }
        __syncthreads();
        u = u_end;
        ++count;
        if (u < units) {
            first += per;
            if (++vh == s.groups * a.c.n_kv_heads) {
                vh = 0;
                do {
                    s = seq_of(a, ++b, ROWS);
                } while (s.groups == 0);
                settle();
                per = seq_units(s);
            }
        }
    }
}

template <int D, int NT>
cudaError_t launch_split(const RopeTable &tab, const AttnArgs &a, cudaStream_t st) {
    using C = Split<D, NT>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_attn_split<D, NT>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    const cudaError_t l = launch_early(k_attn_split<D, NT>, dim3(C::CTAS), kSplitWarps * 32, C::SMEM, st, tab, a);
    return l != cudaSuccess ? l : launch_join<D, C::ROWS, false>(a, C::CTAS, st);
}

}  // namespace

extern "C" size_t strata_kv4_attention_workspace_bytes(const strata_kv4_cache *cache, int32_t n_q_heads) {
    if (strata_check_kv4_cache(cache) != STRATA_OK) return 0;
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads) return 0;
    const size_t split = sizeof(float) * (cache->head_dim + 4) * kSplitParts, tiles = attn_tiles_part_bytes(cache->head_dim);
    return sizeof(Span) * kSplitMaxCtas + (split > tiles ? split : tiles);
}

static strata_status attention(const strata_kv4_cache *cache, const strata_kv4_attn_desc *d, strata_rope rope,
                               const int32_t *positions, const void *q, const int32_t *q_offsets,
                               const int32_t *kv_lens, const int32_t *block_table, void *out, void *workspace,
                               size_t workspace_bytes, const AttnStall *stall, strata_stream_t stream) {
    const strata_status s = strata_check_kv4_cache(cache);
    if (s != STRATA_OK) return s;
    if (!d) return strata_set_error(STRATA_ERR_INVALID_ARG, "NULL desc");
    if (d->n_q_heads < 1 || d->n_q_heads % cache->n_kv_heads)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "n_q_heads %d is not a multiple of n_kv_heads %d", d->n_q_heads,
                                cache->n_kv_heads);
    if (d->n_seqs < 0 || d->n_tokens < 0 || d->max_q_len < 0 || d->max_pages < 0 || d->window < 0)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "a negative count in the desc");
    const float scale_log2 = d->scale * 1.44269504088896340736f;
    if (!std::isfinite(scale_log2)) return strata_set_error(STRATA_ERR_INVALID_ARG, "scale log2(e) is not finite in fp32");
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
               static_cast<__nv_bfloat16 *>(out), workspace, d->n_q_heads / cache->n_kv_heads, 0, 0.f, 0};
    while ((1 << a.page_shift) < cache->page_size) ++a.page_shift;
    a.group_inv = a.group > 1 ? ~0ull / (uint64_t)a.group + 1 : 0;
    a.scale_log2 = scale_log2;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const bool two = (int64_t)d->max_q_len * a.group > 8;
    cudaError_t e;
    if (stall)
        e = launch_attn_tiles_stalled(tab, a, *stall, st);
    else if ((int64_t)d->max_q_len * a.group > kSplitMostRows)
        e = launch_attn_tiles(tab, a, st);
    else if (cache->head_dim == 64)
        e = two ? launch_split<64, 2>(tab, a, st) : launch_split<64, 1>(tab, a, st);
    else if (cache->head_dim == 128)
        e = two ? launch_split<128, 2>(tab, a, st) : launch_split<128, 1>(tab, a, st);
    else
        e = launch_split<256, 1>(tab, a, st);
    if (e != cudaSuccess) return strata_set_error(STRATA_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return STRATA_OK;
}

extern "C" strata_status strata_kv4_attention(const strata_kv4_cache *cache, const strata_kv4_attn_desc *d,
                                              strata_rope rope, const int32_t *positions, const void *q,
                                              const int32_t *q_offsets, const int32_t *kv_lens,
                                              const int32_t *block_table, void *out, void *workspace,
                                              size_t workspace_bytes, strata_stream_t stream) {
    return attention(cache, d, rope, positions, q, q_offsets, kv_lens, block_table, out, workspace, workspace_bytes,
                     nullptr, stream);
}

extern "C" strata_status strata_selftest_attention_timeout(const strata_kv4_cache *cache, const strata_kv4_attn_desc *d,
                                                           const void *q, const int32_t *q_offsets,
                                                           const int32_t *kv_lens, const int32_t *block_table,
                                                           void *out, void *workspace, size_t workspace_bytes,
                                                           int32_t role, int32_t every, int32_t piece,
                                                           strata_stream_t stream) {
    if (role < 0 || role > 3 || every < 1 || piece < 0)
        return strata_set_error(STRATA_ERR_INVALID_ARG, "role %d, every %d, piece %d", role, every, piece);
    const AttnStall stall{role, every, piece};
    return attention(cache, d, nullptr, nullptr, q, q_offsets, kv_lens, block_table, out, workspace, workspace_bytes,
                     &stall, stream);
}
