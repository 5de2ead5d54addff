// kv_attn_tiles.cu -- attention over the paged 4-bit cache for many query rows
// (prompt chunks, long verify steps) on the 5th-generation tensor cores.
//
// An item is a KV head of a sequence and up to 256 of its query rows (token-
// major, the group's heads inside; 128 for head_dim 256) against the keys that
// they see, in tiles of 128 keys (64 for head_dim 256). For each tile
//   8 warps expand the packed rows into fp16 (c - 8) s, keys and values, in
//     shared memory (128-byte swizzle), from registers loaded a tile ahead;
//   1 thread issues S = Q K^T and O += P V (tcgen05; S, P and O in tensor
//     memory, P in the columns of its S);
//   8 warps turn S into P: a thread per row, so that maximum and sum need no
//     exchange between lanes.
// Two S stand in tensor memory, of two 128-row halves of the item; where the
// item has at most 128 rows, of every second key tile instead, each with an O
// of its own, added up at the end (head_dim 256: one O, S of two tiles). So the
// tensor cores work on one while the softmax works on the other. Bound by the
// exponentials (16 a cycle and SM) and the matrix products (4 D multiply-adds
// a score), which take the same time at head_dim 128.
//
// Softmax: weights 2^(x - M + 6), M a row's running maximum, moved only when a
// weight would pass 2^11 (then O is scaled in tensor memory). fp16 range of the
// scales: as long as 32 keys' scales are all below 2^12 with some above 2^-10,
// (c - 8) s is a plain fp16 product. Where not, each of these keys is
// normalised by its own power of two, which the softmax takes back: the key's
// as a factor of its scores, the value's as an exponent added to x.
//
// Work: the key tiles of all items in a row, each item with kHead units in front,
// cut into 148 equal runs, one for each CTA; pieces of an item that several CTAs share go through k_attn_join_planes.
//
// Measured (B200): 8,192 tokens of 32 heads of 128, the last of 32,768 (4 KV
// heads): 4.52 ms, 851 TFLOP/s; head_dim 64 3.65 ms, 528 TFLOP/s; 256 14.0 ms,
// 549 TFLOP/s. At 128 a step of 256 rows and 128 keys takes about 5,000 cycles, of
// which the tensor cores work 2,080 (ncu: 32 % of all cycles for 2,048 tokens at
// 8,192) and the exponentials need 2,048: a chain of product, wait, softmax (2,500
// for a half, two halves at once), wait and product, with two halves in flight.
// Tensor memory has no room for a third. At the launch's 96 registers ptxas
// spills 336 bytes of stores and 624 of loads a thread. What was tried:
//   scores 64 keys at a time in four S, so that products of a half overlap its
//     softmax: 436 us against 400 (2,048 tokens at 8,192), a product of 64 columns
//     reads the query rows twice as often;
//   3 of 8 exponentials as polynomials: 424 against 407 us, issue is as scarce;
//   one thread issuing the products: 480 against 420 us, descriptors then move
//     through vector registers; maximum before the weights instead of a test of
//     the packed weights: 408 against 402 us; registers 128 to 152 for the
//     softmax: the same.
#include "kv_attn.cuh"

namespace strata {
namespace {

constexpr int kThreads = 20 * 32;  // the last three warps only complete a group of four
constexpr int kMmaWarp = 16;
// Tiles whose flags are kept. Those of tile c are written ahead of the wait for its
// buffer, once that for c - 1 has ended: the product of c - 3 is done, so c - 5 is
// weighed, and c - 4 may be at it still.
constexpr int kInfo = 8;

template <int D>
struct Tiles {
    static constexpr int NB = D / 32;
    static constexpr int TK = D == 256 ? 64 : 128;      // keys of a tile
    static constexpr int SLOTS = D == 256 ? 1 : 2;      // O accumulators
    static constexpr int ROWS = 128 * SLOTS;            // of an item
    static constexpr int KV = TK * D * 2;               // bytes of a tile's keys in fp16
    static constexpr int Q = 128 * D * 2;               // of 128 query rows
    static constexpr int PART = D + 4;
    static constexpr int O_COL = 256;                   // tensor memory: S at 0 and 128, then O
    static constexpr int S_STEP = 128;
    static constexpr int KMUL = 0, VE = KMUL + kInfo * TK * 4, VINV = VE + kInfo * TK * 4, FLAGS = VINV + kInfo * TK * 4,
                         FAC = FLAGS + kInfo * 8 * 4, ML = FAC + ROWS * 4, AUX = ML + 128 * 8;
    static constexpr int SMEM = 1024 + SLOTS * Q + 4 * KV + AUX;
    static constexpr int SPLIT = D == 256 ? 2 : 1;      // threads for a row of codes
    static constexpr int NW = NB / SPLIT;               // 16-byte words of codes of a thread: a block each
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(128 * D * 4 <= 4 * KV, "the second O fits the tiles' buffers");
};

// The matrix warp runs as one, so that descriptors stay in uniform registers;
// the instructions themselves are issued by its elected thread.
STRATA_DEV uint32_t elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
STRATA_DEV void umma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate, uint32_t me) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(me)
        : "memory");
}
STRATA_DEV void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate, uint32_t me) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(me)
        : "memory");
}
STRATA_DEV void umma_done(uint64_t *bar, uint32_t me) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(me)
        : "memory");
}
// 32 lanes x 32 bits, 32 consecutive columns per thread
STRATA_DEV void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
STRATA_DEV void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
STRATA_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Waits of a whole warp. The lanes ask together and leave the loop together: what
// follows (.aligned instructions, uniform registers) needs the warp in one piece,
// which lanes that leave a loop one by one do not promise.
template <typename Test>
STRATA_DEV bool warp_poll(Test &&test, volatile int *abort, uint64_t limit_ns) {
    if (__all_sync(kFullMask, test())) return true;
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (__all_sync(kFullMask, test())) return true;
        if ((i & 63u) == 0 && __any_sync(kFullMask, (abort && *abort) || globaltimer() - t0 > limit_ns)) {
            if (abort) *abort = 1;
            return false;
        }
    }
}
template <uint64_t LIMIT>
STRATA_DEV bool warp_wait_for(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return warp_poll([&]() { return mbar_try_wait(bar, parity); }, abort, LIMIT);
}
// until a number in shared memory has come up to `least`
STRATA_DEV bool count_wait(volatile uint32_t *count, uint32_t least, volatile int *abort, uint64_t limit_ns) {
    const bool ok = warp_poll([&]() { return *count >= least; }, abort, limit_ns);
    __threadfence_block();
    return ok;
}
// barrier of `threads` threads; whether any of them says stop
STRATA_DEV bool named_barrier_or(int id, int threads, bool stop) {
    uint32_t any;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(any)
        : "r"(id), "r"(threads), "r"((uint32_t)stop)
        : "memory");
    return any != 0;
}
STRATA_DEV void named_barrier(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// Operand with the other dimension contiguous (V: 64 values of a key, 128-byte
// swizzle): groups of 8 keys 1024 bytes apart, blocks of 64 values `block` apart.
STRATA_DEV uint64_t umma_desc_sw128_mn(const void *tile, uint32_t block) {
    uint64_t a = smem_u32(tile);
    return ((a >> 4) & 0x3FFFull) | ((uint64_t)(block >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// Registers of a group of four warps. 640 threads at 96 each are 480 for every
// four-warp column; afterwards 2 x 136 + 2 x 72 + 64 = 480.
template <int N>
STRATA_DEV void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
STRATA_DEV void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

STRATA_DEV uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
STRATA_DEV float2 unpack2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
STRATA_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
STRATA_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
STRATA_DEV uint32_t and_or(uint32_t w, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
    return r;
}
STRATA_DEV uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
STRATA_DEV __half2 bits_h2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }

// Tiles of keys, values and query rows: blocks of 64 values, rows of 128 bytes in
// 16-byte chunks of 8 values, chunk c of row r at c ^ (r & 7) (128-byte swizzle).
// Inside 8 values the chunks hold 0 4 1 5 2 6 3 7: the order of a code word's nibble pairs
__host__ __device__ constexpr int place_of(int n) { return n < 4 ? 2 * n : 2 * n - 7; }
__host__ __device__ constexpr int value_at(int p) { return p & 1 ? 4 + (p >> 1) : p >> 1; }

struct Item {  // up to ROWS query rows of a KV head
    int rows, row0, tile0, tiles;  // key tiles
};
template <int D>
STRATA_DEV Item item_of(const AttnArgs &a, const SeqBase &s, int rt) {
    using C = Tiles<D>;
    Item it;
    it.row0 = rt * C::ROWS;
    it.rows = min(C::ROWS, s.n * a.group - it.row0);
    const int first = by_group(a, it.row0), last = by_group(a, it.row0 + it.rows - 1);
    const int hi = max(s.L - s.n + last + 1, 0);
    const int lo = a.d.window > 0 ? (int)max((int64_t)0, (int64_t)s.L - s.n + first - a.d.window + 1) : 0;
    it.tile0 = min(lo, hi) / C::TK;
    it.tiles = (int)(((int64_t)hi + C::TK - 1) / C::TK) - it.tile0;
    return it;
}
// Units of an item: those that stand for what a piece of it costs besides its
// tiles (rows in, results out), then its tiles; one at least, which writes the
// zeros of rows without keys.
// us with 0, 3, 6, 10 (head_dim 128, the first 64): mixed batch 65, 60, 59, 58; 4 sequences of 512 tokens up to
// 4,096 118, 114, 109, 120; 8 of 16 up to 16,000 137, 111, 89, 89; 3 of 1,500 with
// a window of 512 146, 124, 134, 141.
constexpr int kHead = 8;
STRATA_DEV int item_units(const Item &it) { return kHead + max(it.tiles, 1); }

// A run of a CTA's key tiles inside one item, and what came before it
struct Piece {
    int b, hk, rt, first, u, u_end;  // units count from the CTA's first; first: of the item
    SeqBase s;
    Item it;
    int kt0, nt, steps;
    bool whole, dual, after_dual;
    uint32_t tc, sc[2], count;  // key tiles, steps in each S, pieces so far: buffers and phases
};

// Where a CTA leaves a partial result: its first piece may go on from the CTA
// before it, its last one into the next
STRATA_DEV int slot_of(const Piece &p) { return p.count ? 1 : 0; }

STRATA_DEV int item_count(const AttnArgs &a, int n, int rows) { return (int)(((int64_t)n * a.group + rows - 1) / rows); }

// Units of one KV head of a sequence, by a whole warp
template <int D>
STRATA_DEV int64_t head_units(const AttnArgs &a, const SeqBase &s, int lane) {
    const int count = item_count(a, s.n, Tiles<D>::ROWS);
    int64_t v = 0;
    for (int rt = lane; rt < count; rt += 32) v += item_units(item_of<D>(a, s, rt));
#pragma unroll
    for (int x = 16; x; x >>= 1) v += __shfl_xor_sync(kFullMask, v, x);
    return v;
}

// STALL: the self test of waits that run out, with a limit of its own. Where one
// does, everybody else in the CTA gives up soon after, and the softmax warps make
// every row that this CTA still owes NaN: those of the piece at hand, and without
// another wait those of the pieces behind it. A row that a broken CTA has a part
// of cannot pass for a result.
template <int D, bool STALL>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_tiles(const __grid_constant__ RopeTable tab, const __grid_constant__ AttnArgs a,
                 const __grid_constant__ AttnStall stall) {
    using C = Tiles<D>;
    constexpr uint64_t kLimitNs = STALL ? 5000000ull : kWaitLimitNs;
    auto warp_wait = [](uint64_t *bar, uint32_t parity, volatile int *abort) {
        return warp_wait_for<kLimitNs>(bar, parity, abort);
    };
    auto arrives = [&](int role, uint32_t piece) {
        return !STALL || role != stall.role || blockIdx.x % stall.every != 0 || piece < (uint32_t)stall.piece;
    };
    constexpr int NB = C::NB, TK = C::TK, P = D / 32, SLOTS = C::SLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sq = smem, *sk = sq + SLOTS * C::Q, *sv = sk + 2 * C::KV, *aux = sv + 2 * C::KV;
    float *kmul = reinterpret_cast<float *>(aux + C::KMUL), *ve = reinterpret_cast<float *>(aux + C::VE),
          *vinv = reinterpret_cast<float *>(aux + C::VINV), *sfac = reinterpret_cast<float *>(aux + C::FAC);
    uint32_t *flags = reinterpret_cast<uint32_t *>(aux + C::FLAGS);  // [kInfo][4 groups of 32 keys](holes, slow)
    float2 *sml = reinterpret_cast<float2 *>(aux + C::ML);
    __shared__ uint64_t kfull[2], vfull[2], kempty[2], vempty[2], sfull[2], pready[2], pvdone, odone, qfull;
    __shared__ uint32_t tmem_base;
    __shared__ int s_abort, s_b;
    __shared__ uint32_t s_begun;  // pieces whose rows are there: the results of those before are out
    __shared__ int64_t s_sum[kThreads / 32], s_before;
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    griddep_launch_dependents();

    // rows that no item fills stay finite
    for (int i = threadIdx.x; i < SLOTS * C::Q / 16; i += kThreads) reinterpret_cast<uint4 *>(sq)[i] = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < C::ROWS; i += kThreads) sfac[i] = 1.f;
    fence_proxy_async_smem();
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&kfull[i], 4);
            mbar_init(&vfull[i], 4);
            mbar_init(&kempty[i], 1);
            mbar_init(&vempty[i], 1);
            mbar_init(&sfull[i], 1);
            mbar_init(&pready[i], 4);
        }
        mbar_init(&pvdone, 1);
        mbar_init(&odone, 1);
        mbar_init(&qfull, 8);
        s_abort = 0;
        s_begun = 0;
        fence_mbar_init();
    }

    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    griddep_wait();

    // ---- this CTA's run of units, and the item that it starts in
    int64_t run = 0, inc = 0, v = 0;
    // the units of 32 sequences, by a whole warp; inc: up to and with b0 + lane
    auto scan32 = [&](int b0, SeqBase &s) {
        const int b = b0 + lane;
        v = 0;
        s = SeqBase{0, 0, 0};
        if (b < a.d.n_seqs) load_seq(s, a, b);
        const int count = item_count(a, s.n, C::ROWS);
        for (int rt = 0; rt < count && count <= 4; ++rt) v += item_units(item_of<D>(a, s, rt));
        for (uint32_t many = __ballot_sync(kFullMask, count > 4); many; many &= many - 1) {
            const int src = __ffs(many) - 1;  // long prompts: the lanes together
            const SeqBase o{0, __shfl_sync(kFullMask, s.n, src), __shfl_sync(kFullMask, s.L, src)};
            const int64_t sum = head_units<D>(a, o, lane);
            if (lane == src) v = sum;
        }
        v *= a.c.n_kv_heads;
        inc = v;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int64_t o = __shfl_up_sync(kFullMask, inc, x);
            if (lane >= x) inc += o;
        }
    };
    auto scan = [&](int b0) {  // the same by the block; run: with the whole chunk
        SeqBase s;
        scan32(b0 + warp * 32, s);
        if (lane == 31) s_sum[warp] = inc;
        __syncthreads();
        inc += run;
        for (int w = 0; w < kThreads / 32; ++w) {
            const int64_t o = s_sum[w];
            if (w < warp) inc += o;
            run += o;
        }
        __syncthreads();
    };
    // Up to 32 sequences: every warp for itself
    const bool few = a.d.n_seqs <= 32;
    SeqBase s{0, 0, 0};
    if (few) {
        scan32(0, s);
        run = __shfl_sync(kFullMask, inc, 31);
    } else {
        for (int b0 = 0; b0 < a.d.n_seqs; b0 += kThreads) scan(b0);
    }
    const int64_t total = run;
    const int ctas = (int)min(total, (int64_t)kSms);  // a unit each at least
    Span *spans = static_cast<Span *>(a.workspace);
    float *parts = reinterpret_cast<float *>(spans + kSplitMaxCtas);
    if (threadIdx.x == 0) spans[blockIdx.x].parts = 0;
    const bool idle = blockIdx.x >= ctas;
    const int64_t u_lo = idle ? 0 : run_start(total, blockIdx.x, ctas), u_hi = idle ? 0 : run_start(total, blockIdx.x + 1, ctas);
    if (!few && !idle) {
        int b0 = 0;
        if (a.d.n_seqs > kThreads) {
            run = 0;
            for (b0 = -kThreads; run <= u_lo;) scan(b0 += kThreads);
        }
        if (inc - v <= u_lo && u_lo < inc) {
            s_b = b0 + threadIdx.x;
            s_before = inc - v;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_base;
    if (idle) {
        if (warp == kMmaWarp) tmem_dealloc(tbase, 512);
        return;
    }

    int b, hk = 0, rt = 0, first;  // units count from u_lo; first: of the item
    int64_t before;
    if (few) {
        b = __ffs(__ballot_sync(kFullMask, u_lo < inc)) - 1;
        before = __shfl_sync(kFullMask, inc - v, b);
        s = SeqBase{__shfl_sync(kFullMask, s.t0, b), __shfl_sync(kFullMask, s.n, b), __shfl_sync(kFullMask, s.L, b)};
    } else {
        b = uniform(s_b);
        before = s_before;
        load_seq(s, a, b);
    }
    Item it;
    {
        const int64_t per = head_units<D>(a, s, lane);
        hk = uniform((int)run_start(u_lo - before, 1, per));
        int64_t rem = u_lo - before - hk * per;
        for (;; rt += 32) {  // the item that holds unit `rem`
            const int n = rt + lane < item_count(a, s.n, C::ROWS) ? item_units(item_of<D>(a, s, rt + lane)) : 0;
            int64_t upto = n;
#pragma unroll
            for (int x = 1; x < 32; x <<= 1) {
                const int64_t o = __shfl_up_sync(kFullMask, upto, x);
                if (lane >= x) upto += o;
            }
            const uint32_t past = __ballot_sync(kFullMask, upto > rem);
            if (past) {
                const int src = __ffs(past) - 1;
                rt += src;
                first = -(int)(rem - __shfl_sync(kFullMask, upto - n, src));
                break;
            }
            rem -= __shfl_sync(kFullMask, upto, 31);
        }
        it = item_of<D>(a, s, rt);
    }
    const int units = (int)(u_hi - u_lo);
    const uint32_t n_pages = (uint32_t)min(a.c.n_pages, (int64_t)0x80000000);

    // Every role walks over the pieces by itself, with its own registers.
    auto pieces = [&](auto &&role) {
    Piece p{};
    p.b = b, p.hk = hk, p.rt = rt, p.first = first, p.s = s, p.it = it;
    for (; p.u < units;) {
        const int per = item_units(p.it);
        p.u_end = min(p.first + per, units);
        const int t_lo = max(p.u - p.first - kHead, 0), t_hi = p.u_end - p.first - kHead;
        if (t_hi <= t_lo) break;  // the run ends before the item's first tile
        p.whole = t_lo == 0 && p.u_end == p.first + per;
        p.kt0 = p.it.tile0 + t_lo;
        p.nt = min(t_hi, p.it.tiles) - t_lo;  // 0: rows without keys
        p.dual = SLOTS == 2 && p.it.rows <= 128;
        p.steps = SLOTS == 2 && !p.dual ? 2 * p.nt : p.nt;

        if (!role(p)) break;
        // ---- the next piece
        if (t_lo == 0 && !p.whole && threadIdx.x == 0) {
            // it starts here and ends in the CTA that holds its last unit
            const int64_t last = u_lo + p.first + per - 1;
            int c = (int)run_start(ctas, last, total);  // run c starts at `last` or before it
            while (run_start(total, c + 1, ctas) <= last) ++c;
            spans[blockIdx.x] = Span{c - (int)blockIdx.x + 1, slot_of(p), (int)p.s.t0, p.it.rows, p.hk, p.it.row0, {0, 0}};
        }
        p.tc += p.nt;
        if (SLOTS == 2)
            p.sc[0] += p.dual ? (p.nt + 1) / 2 : p.nt, p.sc[1] += p.dual ? p.nt / 2 : p.nt;
        else
            p.sc[0] += (p.nt + 1) / 2, p.sc[1] += p.nt / 2;
        ++p.count;
        if (p.nt > 0) p.after_dual = p.dual;
        p.u = p.u_end;
        if (p.u < units) {
            p.first += per;
            if (++p.rt == item_count(a, p.s.n, C::ROWS)) {
                p.rt = 0;
                if (++p.hk == a.c.n_kv_heads) {
                    p.hk = 0;
                    do {
                        load_seq(p.s, a, ++p.b);
                    } while (p.s.n == 0);
                }
            }
            p.it = item_of<D>(a, p.s, p.rt);
        }
    }
    };

    if (warp >= kMmaWarp) {
        regs_down<64>();
        const uint32_t me = elected();
        if (warp == kMmaWarp) pieces([&](const Piece &p) {
            // ------------------------------------------------ matrix products
            constexpr uint32_t idesc_s = umma_idesc_f16(128, TK), idesc_o = umma_idesc_f16(128, D) | (1u << 16);
            const bool pairs = SLOTS == 2 && !uniform(p.dual);  // two steps for each key tile
            const int steps = uniform(p.steps);
            const bool shifted = uniform(p.dual && p.it.rows <= 64);
            const uint32_t tc = uniform(p.tc), sc[2] = {(uint32_t)uniform(p.sc[0]), (uint32_t)uniform(p.sc[1])};
            // the rows are there, and what the last piece left in tensor memory has been read
            bool ok = warp_wait(&qfull, p.count & 1, &s_abort);
            tc_fence_after();
            auto product_s = [&](int n) {
                const uint32_t c = tc + (pairs ? n >> 1 : n), i = n & 1;
                if (!warp_wait(&kfull[c & 1], (c >> 1) & 1, &s_abort)) return false;
                tc_fence_after();
                const uint64_t qd = umma_desc_sw128(sq + (pairs || shifted ? i : 0) * C::Q), kd = umma_desc_sw128(sk + (c & 1) * C::KV);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    umma_ss(tbase + i * C::S_STEP, qd + (k >> 2) * (128 * 128 / 16) + (k & 3) * 2,
                            kd + (k >> 2) * (TK * 128 / 16) + (k & 3) * 2, idesc_s, k ? 1u : 0u, me);
                umma_done(&sfull[i], me);
                if (!pairs || i) umma_done(&kempty[c & 1], me);
                return true;
            };
            for (int n = 0; n < 2 && n < steps && ok; ++n) ok = product_s(n);
            for (int n = 0; n < steps && ok; ++n) {
                const uint32_t c = tc + (pairs ? n >> 1 : n), i = n & 1;
                ok = warp_wait(&vfull[c & 1], (c >> 1) & 1, &s_abort) &&
                     warp_wait(&pready[i], (sc[i] + (n >> 1)) & 1, &s_abort);
                if (!ok) break;
                tc_fence_after();
                const uint64_t vd = umma_desc_sw128_mn(sv + (c & 1) * C::KV, TK * 128);
                const uint32_t more = (SLOTS == 2 ? n >= 2 : n >= 1) ? 1u : 0u;
#pragma unroll
                for (int k = 0; k < TK / 16; ++k)
                    umma_ts(tbase + C::O_COL + (SLOTS == 2 ? i * D : 0), tbase + i * C::S_STEP + k * 8,
                            vd + k * (2048 / 16), idesc_o, k ? 1u : more, me);
                if (SLOTS == 1) umma_done(&pvdone, me);
                if (!pairs || i) umma_done(&vempty[c & 1], me);
                if (n + 2 < steps) ok = product_s(n + 2);
            }
            if (!ok) __threadfence_block();  // who sees this barrier sees s_abort
            umma_done(&odone, me);
            warp_wait(&odone, p.count & 1, nullptr);  // before anything is torn down
            return ok;
        });
    } else if (warp >= 8) {
        regs_down<72>();
        pieces([&](const Piece &p) {
            // ------------------------------------------------ expanding keys (warps 8-11) and values (12-15)
            const bool is_v = warp >= 12;
            const int id = threadIdx.x - (is_v ? 384 : 256), row = id % TK, part = id / TK;
            const int32_t *table = a.table + (int64_t)p.b * a.d.max_pages;
            const uint8_t *codes = static_cast<const uint8_t *>(is_v ? a.c.v_codes : a.c.k_codes) + part * (C::NW * 16);
            const uint8_t *vsc = static_cast<const uint8_t *>(a.c.v_scales), *ksc = static_cast<const uint8_t *>(a.c.k_scales);
            // what no row of the item sees is not read: it may hold anything
            const int pos0 = p.s.L - p.s.n, any_hi = min(pos0 + by_group(a, p.it.row0 + p.it.rows - 1) + 1, p.s.L);
            const int any_lo = a.d.window > 0 ? (int)max((int64_t)pos0 + by_group(a, p.it.row0) - a.d.window, (int64_t)-1) : -1;
            uint32_t page = ~0u;
            auto find = [&](int jj) {  // the page of this thread's key in tile jj
                const int64_t key = (int64_t)(p.kt0 + jj) * TK + row;
                page = jj < p.nt && key < any_hi && key > any_lo ? (uint32_t)__ldg(table + (key >> a.page_shift)) : ~0u;
            };
            uint4 w[C::NW];
            uint32_t vs[NB / 2], ks[NB / 2];
            bool here = false;
            auto load = [&](int jj) {
                here = page < n_pages;
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) vs[i] = ks[i] = 0u;
#pragma unroll
                for (int i = 0; i < C::NW; ++i) w[i] = make_uint4(0, 0, 0, 0);
                if (here) {
                    const int slot = (int)(((int64_t)(p.kt0 + jj) * TK + row) & (a.c.page_size - 1));
                    const uint64_t at = ((page * a.c.n_kv_heads + p.hk) << a.page_shift) + (uint32_t)slot;
#pragma unroll
                    for (int i = 0; i < C::NW; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(codes + at * (D / 2)) + i);
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) {
                        vs[i] = __ldg(reinterpret_cast<const uint32_t *>(vsc + at * (D / 16)) + i);
                        if (!is_v) ks[i] = __ldg(reinterpret_cast<const uint32_t *>(ksc + at * (D / 16)) + i);
                    }
                }
            };
            find(0);
            load(0);
            find(1);
            // The second O of the last dual piece was added up in the keys' buffers. These
            // warps may be pieces ahead, where a barrier's parity says nothing: a count.
            if (p.nt > 0 && p.after_dual && !count_wait(&s_begun, p.count + 1, &s_abort, kLimitNs)) return false;
            for (int jj = 0; jj < p.nt; ++jj) {
                const uint32_t c = p.tc + jj;
                // the scales' ranges decide for 32 keys at a time; keys and values see the same numbers
                auto range = [&](const uint32_t (&x)[NB / 2], uint32_t &top) {
                    uint32_t m = 0;
#pragma unroll
                    for (int i = 0; i < NB / 2; ++i) m = max(m, max(x[i] << 17, (x[i] & 0x7fff0000u) << 1));
                    top = m >> 17;
                    return __any_sync(kFullMask, m >= 0x6c00u << 17) || !__any_sync(kFullMask, m >= 0x1400u << 17);
                };
                uint32_t vtop, ktop = 0;
                const bool v_slow = range(vs, vtop), k_slow = !is_v && range(ks, ktop);
                const int ev = (int)max(vtop >> 10, 1u) - 16, ek = (int)max(ktop >> 10, 1u) - 16;  // s 2^-e in [2, 4)
                if (!is_v && part == 0) {
                    const int info = c & (kInfo - 1);
                    const uint32_t holes = __ballot_sync(kFullMask, !here && (int64_t)(p.kt0 + jj) * TK + row < p.s.L);
                    if (lane == 0) {
                        flags[info * 8 + (row >> 5) * 2] = holes;
                        flags[info * 8 + (row >> 5) * 2 + 1] = (k_slow ? 1u : 0u) | (v_slow ? 2u : 0u);
                    }
                    if (k_slow || v_slow) {
                        kmul[info * TK + row] = k_slow ? __int_as_float((127 + ek) << 23) : 1.f;
                        ve[info * TK + row] = v_slow ? (float)ev : 0.f;
                        vinv[info * TK + row] = v_slow ? __int_as_float((127 - ev) << 23) : 1.f;
                    }
                }
                const bool slow = is_v ? v_slow : k_slow;
                const int e = is_v ? ev : ek;
                uint4 cw[C::NW];
                uint32_t cs[C::NW];
#pragma unroll
                for (int i = 0; i < C::NW; ++i) {
                    cw[i] = w[i];
                    const int k = part * C::NW + i;
                    const uint32_t x = is_v ? (NB > 4 ? (part ? vs[2 + i / 2] : vs[i / 2]) : vs[i / 2])
                                            : (NB > 4 ? (part ? ks[2 + i / 2] : ks[i / 2]) : ks[i / 2]);
                    cs[i] = __byte_perm(x, 0, (k & 1) ? 0x3232 : 0x1010);
                }
                load(jj + 1);
                find(jj + 2);
                uint64_t *full = is_v ? &vfull[c & 1] : &kfull[c & 1], *empty = is_v ? &vempty[c & 1] : &kempty[c & 1];
                if (!warp_wait(empty, ((c >> 1) & 1) ^ 1, &s_abort)) return false;
                const uint32_t to = smem_u32((is_v ? sv : sk) + (c & 1) * C::KV) + row * 128 + ((row & 7) << 4);  // chunk 0
                if (slow) {
                    const __half2 mul = bits_h2((uint32_t)(15 - e) * 0x04000400u);  // 2^-e, -15 <= e <= 14
#pragma unroll
                    for (int i = 0; i < C::NW; ++i) cs[i] = h2_bits(__hmul2(bits_h2(cs[i]), mul));
                }
                const __half2 off = __floats2half2_rn(-1032.f, -1032.f), off64 = __floats2half2_rn(-72.f, -72.f);
#pragma unroll
                for (int i = 0; i < C::NW; ++i) {
                    const uint32_t words[4] = {cw[i].x, cw[i].y, cw[i].z, cw[i].w};
                    const __half2 sc2 = bits_h2(cs[i]);
                    const uint32_t at = (to ^ ((i & 1) << 6)) + (part * (C::NW / 2) + (i >> 1)) * (TK * 128);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t x = words[j], y = x >> 8;
                        uint4 o;
                        o.x = h2_bits(__hmul2(__hadd2(bits_h2(and_or(x, 0x000f000fu, 0x64006400u)), off), sc2));
                        o.y = h2_bits(__hmul2(__hadd2(bits_h2(and_or(x, 0x00f000f0u, 0x54005400u)), off64), sc2));
                        o.z = h2_bits(__hmul2(__hadd2(bits_h2(and_or(y, 0x000f000fu, 0x64006400u)), off), sc2));
                        o.w = h2_bits(__hmul2(__hadd2(bits_h2(and_or(y, 0x00f000f0u, 0x54005400u)), off64), sc2));
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ (j << 4)), "r"(o.x), "r"(o.y),
                                     "r"(o.z), "r"(o.w)
                                     : "memory");
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && arrives(is_v ? 1 : 0, p.count)) mbar_arrive(full);
            }
            return true;
        });
    } else {
        regs_up<136>();
        pieces([&](const Piece &p) {
        auto tile_of = [&](int n) { return SLOTS == 2 && !p.dual ? n >> 1 : n; };  // of step n, in S n & 1
            // ------------------------------------------------ softmax: S slot (warps 0-3, 4-7), a thread per row
            // the rows first: rotary, transform, fp16 with a power-of-two scale; a warp
            // takes rows in a run, which share a token's angles
            {
                using Q = QueryRow<D>;
                if (p.count) named_barrier(3, 256);  // the last piece's results went through the rows' place
                const int shift = p.dual && p.it.rows <= 64 ? 64 : 0;
                constexpr int BATCH = 2;
                const int run = (min(p.it.rows, p.dual || SLOTS == 1 ? 128 : 256) + 7) / 8;  // 32 at most
                const int end = min(warp * run + run, p.it.rows), first_row = warp * run;
                // a lane for each row of the run: its place and its token's position
                const int my_row = p.it.row0 + min(first_row + lane, p.it.rows - 1), my_tok = by_group(a, my_row);
                const int64_t my_at = (p.s.t0 + my_tok) * a.d.q_token_stride +
                                      (int64_t)(p.hk * a.group + my_row - my_tok * a.group) * D;
                const int my_pos = tab.rd ? a.positions[p.s.t0 + my_tok] : 0;
                const int chunk = (lane * P >> 3) & 7;  // of the row, in its block of 64 values
                const uint32_t place = smem_u32(sq) + (lane * P >> 6) * (128 * 128) + place_of(lane * P & 7) * 2;
                float2 cs[P];
                int at = -1;
                typename Q::Raw raw[BATCH], next[BATCH];
                auto fetch = [&](int r0) {
#pragma unroll
                    for (int k = 0; k < BATCH; ++k)
                        Q::load(next[k], a.q + __shfl_sync(kFullMask, my_at, min(r0 + k - first_row, 31)), tab, lane);
                };
                fetch(first_row);
#pragma unroll 1
                for (int r0 = first_row; r0 < end; r0 += BATCH) {
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) raw[k] = next[k];
                    fetch(r0 + BATCH);
                    float q[BATCH][P], m[BATCH];
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {  // past the end: the last row once more
                        const int r = min(r0 + k, end - 1) - first_row, tok = __shfl_sync(kFullMask, my_tok, r);
                        if (tok != at) {
                            at = tok;
                            Q::angles(cs, tab, __shfl_sync(kFullMask, my_pos, r), lane);
                        }
                        Q::rotate(q[k], raw[k], cs, tab, lane);
                    }
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        fwht_warp<D>(q[k], lane);
                        m[k] = 0.f;
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            q[k][i] *= a.scale_log2 < 0.f ? -rsqrt_dim<D>() : rsqrt_dim<D>();
                            m[k] = fmaxf(m[k], fabsf(q[k][i]));
                        }
                    }
#pragma unroll
                    for (int x = 16; x; x >>= 1)
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) m[k] = fmaxf(m[k], __shfl_xor_sync(kFullMask, m[k], x));
#pragma unroll
                    for (int k = 0; k < BATCH; ++k) {
                        const int r = r0 + k;
                        if (r >= end) break;  // what lies behind keeps older rows' values: never stored
                        const uint32_t ex = min(max(__float_as_uint(m[k]) >> 23, 1u), 252u);
                        const float mul = m[k] > 0.f ? __uint_as_float((253u - ex) << 23) : 1.f;  // largest value to [0.5, 1)
                        const uint32_t to = place + (r >> 7) * C::Q + (r & 127) * 128 + ((chunk ^ (r & 7)) << 4);
#pragma unroll
                        for (int i = 0; i < P; ++i) {  // P <= 4: the lane's values are every second one of its chunk
                            const uint16_t x = __half_as_ushort(__float2half_rn(q[k][i] * mul));
                            const uint32_t off = P == 8 ? place_of(i) * 2 : 4 * i;
                            asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + off), "h"(x) : "memory");
                            if (shift) asm volatile("st.shared.b16 [%0], %1;" ::"r"(to + off + C::Q + 64 * 128), "h"(x) : "memory");
                        }
                        // above zero, so that a masked score stays -inf
                        if (lane == 0)
                            sfac[r] = fmaxf(fabsf(a.scale_log2) * (m[k] > 0.f ? __uint_as_float((ex + 1) << 23) : 1.f), 1e-37f);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                // the factors are read by other warps; after a wait that ran out all of them only mark their rows
                if (named_barrier_or(2, 256, *(volatile int *)&s_abort != 0)) {
                    if (p.whole) {
                        for (int i = threadIdx.x; i < p.it.rows * (D / 8); i += 256) {
                            const int row = p.it.row0 + i / (D / 8), tok = by_group(a, row);
                            const int h = p.hk * a.group + row - tok * a.group;
                            *reinterpret_cast<uint4 *>(a.out + (p.s.t0 + tok) * a.d.out_token_stride + (int64_t)h * D +
                                                       i % (D / 8) * 8) =
                                make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
                        }
                    } else {
                        float4 *part = reinterpret_cast<float4 *>(parts + (int64_t)(blockIdx.x * 2 + slot_of(p)) * C::ROWS * C::PART);
                        for (int i = threadIdx.x; i < (D / 4 + 1) * C::ROWS; i += 256) part[i] = make_float4(NAN, NAN, NAN, NAN);
                    }
                    return true;
                }
                if (threadIdx.x == 0) {
                    __threadfence_block();
                    *(volatile uint32_t *)&s_begun = p.count + 1;
                }
                if (lane == 0 && arrives(3, p.count)) mbar_arrive(&qfull);
            }
            const int slot = warp >> 2, tr = threadIdx.x & 127;
            const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
            const uint32_t ocol = lanes + C::O_COL + (SLOTS == 2 ? slot * D : 0);
            // At most 64 rows against alternate tiles: the second S has them in the
            // other half of tensor memory, for the warps of the other two schedulers.
            const int shift = p.dual && p.it.rows <= 64 ? 64 * slot : 0;
            const int r = (SLOTS == 2 && !p.dual ? slot * 128 : 0) + tr - shift;  // of the item; outside it: no row
            const bool busy = __any_sync(kFullMask, r >= 0 && r < p.it.rows);
            const int pos = p.s.L - p.s.n + by_group(a, p.it.row0 + min(max(r, 0), p.it.rows - 1));
            const int hi = min(pos, p.s.L - 1), lo = a.d.window > 0 ? (int)max((int64_t)pos - a.d.window, (int64_t)-1) : -1;
            const int full_hi = p.s.L - p.s.n + by_group(a, p.it.row0);
            const int full_lo =
                a.d.window > 0 ? (int)max((int64_t)p.s.L - p.s.n + by_group(a, p.it.row0 + p.it.rows - 1) - a.d.window, (int64_t)-1) : -1;
            const float fac = sfac[max(r, 0)];
            float M = -FLT_MAX, l = 0.f;
            uint32_t n_s[2] = {p.sc[0], p.sc[1]};
            bool ok = true;
            int mine = 0;  // p.steps of this slot
            for (int n = slot; n < p.steps && slot < SLOTS; n += SLOTS, ++mine) {
                const int i = SLOTS == 2 ? slot : n & 1;
                const int jj = tile_of(n), k0 = (p.kt0 + jj) * TK, info = (p.tc + jj) & (kInfo - 1);
                ok = warp_wait(&sfull[i], n_s[i] & 1, &s_abort);
                if (!ok) break;
                ++n_s[i];
                if (!busy) {  // P of rows that are not there may be anything
                    if (lane == 0) mbar_arrive(&pready[i]);
                    continue;
                }
                tc_fence_after();
                const uint32_t scol = lanes + i * C::S_STEP;
                float xa[32];
                tmem_ld32(scol, xa);
                uint32_t slow = 0, any = 0;
#pragma unroll
                for (int g = 0; g < TK / 32; ++g) {
                    const uint2 f = *reinterpret_cast<const uint2 *>(flags + info * 8 + g * 2);
                    any |= f.x;
                    slow |= f.y;
                }
                const bool plain = k0 + TK - 1 <= full_hi && k0 > full_lo && any == 0;
                uint64_t sum[2] = {0, 0};
                // M moves by whole numbers: what was computed with the old one (chunks before g, O) is scaled exactly
                auto move = [&](float top, int g) {
                    const float m = fmaxf(M, ceilf(top - 6.f)), f = ex2(M - m);
                    M = m;
                    l *= f;
                    const uint64_t ff = pack2(f, f);
                    sum[0] = fma2(sum[0], ff, 0), sum[1] = fma2(sum[1], ff, 0);
                    const __half2 fh = __float2half2_rn(f);
                    tmem_st_wait();  // what this step has stored so far is read back
#pragma unroll 1
                    for (int h = 0; h < g; ++h) {
                        float y[16];
                        uint32_t w[16];
                        tmem_ld16(scol + 16 * h, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = h2_bits(__hmul2(bits_h2(__float_as_uint(y[e])), fh));
                        tmem_st16(scol + 16 * h, w);
                    }
                    if (!mine) return;
                    if (SLOTS == 1) {  // the last product may still run: S of this step was issued before it
                        ok = warp_wait(&pvdone, (p.tc + n - 1) & 1, &s_abort) && ok;
                        tc_fence_after();
                    }
#pragma unroll 1
                    for (int h = 0; h < D / 16; ++h) {
                        float y[16];
                        uint32_t w[16];
                        tmem_ld16(ocol + 16 * h, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(y[e] * f);
                        tmem_st16(ocol + 16 * h, w);
                    }
                };
                auto largest = [&](const float (&x)[32]) {
                    float t[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        t[k] = fmaxf(x[8 * k], x[8 * k + 1]);
#pragma unroll
                        for (int e = 2; e < 8; e += 2) t[k] = fmaxf(fmaxf(t[k], x[8 * k + e]), x[8 * k + e + 1]);
                    }
                    return fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
                };
                auto weigh = [&](const float (&x)[32], float (&w)[32], float fg) {
                    const uint64_t f2 = pack2(fg, fg), m2 = pack2(-M, -M);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 z = unpack2(fma2(pack2(x[e], x[e + 1]), f2, m2));
                        w[e] = ex2(z.x), w[e + 1] = ex2(z.y);
                    }
                };
                // The same with x fg rounded first, as it was for the maximum: of logits from
                // 2^27 on, fp32 numbers lie so far apart that the unrounded product can pass
                // M by more than fp16 holds, or stay behind it by as much.
                auto weigh_rounded = [&](const float (&x)[32], float (&w)[32], float fg) {
                    const uint64_t f2 = pack2(fg, fg), m2 = pack2(-M, -M);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        const float2 z = unpack2(add2(fma2(pack2(x[e], x[e + 1]), f2, 0), m2));
                        w[e] = ex2(z.x), w[e + 1] = ex2(z.y);
                    }
                };
                auto pack = [&](const float (&w)[32], uint32_t (&y)[16]) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) y[e] = h2_bits(__floats2half2_rn(w[2 * e], w[2 * e + 1]));
                };
                auto add = [&](const float (&x)[32]) {
#pragma unroll
                    for (int e = 0; e < 32; e += 2) sum[e / 2 & 1] = add2(sum[e / 2 & 1], pack2(x[e], x[e + 1]));
                };
                if (plain && slow == 0) {
                    // the weights themselves tell, as fp16, whether M has to move first
#pragma unroll 2
                    for (int g = 0; g < TK / 32; ++g) {
                        float w[32];
                        uint32_t y[16];
                        tmem_ld_wait();
                        weigh(xa, w, fac);
                        if (g + 1 < TK / 32) tmem_ld32(scol + 32 * g + 32, xa);  // comes up meanwhile
                        pack(w, y);
                        __half2 t[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            t[k] = __hmax2(__hmax2(bits_h2(y[4 * k]), bits_h2(y[4 * k + 1])),
                                           __hmax2(bits_h2(y[4 * k + 2]), bits_h2(y[4 * k + 3])));
                        const uint32_t m = h2_bits(__hmax2(__hmax2(t[0], t[1]), __hmax2(t[2], t[3])));
                        if (__any_sync(kFullMask, max(m >> 16, m & 0xffffu) > 0x6800u)) {  // 2^11
                            tmem_ld32(scol + 32 * g, w);
                            tmem_ld_wait();  // ends the load ahead too
                            move(largest(w) * fac, g);
                            weigh_rounded(w, w, fac);
                            pack(w, y);
                        }
                        tmem_st16(scol + 16 * g, y);  // columns that were read before
                        add(w);
                    }
                } else {
                    tmem_ld_wait();
#pragma unroll 1
                    for (int g = 0; g < TK / 32; ++g) {
                        float x[32];
                        tmem_ld32(scol + 32 * g, x);
                        tmem_ld_wait();
                        const bool own = flags[info * 8 + g * 2 + 1] != 0;
                        const float fg = own ? 1.f : fac;
                        if (own) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                x[e] = fmaf(x[e] * kmul[info * TK + 32 * g + e], fac, ve[info * TK + 32 * g + e]);
                        }
                        const int c0 = k0 + 32 * g;
                        const uint32_t hole = flags[info * 8 + g * 2];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c0 + e > hi || c0 + e <= lo || (hole >> e & 1)) x[e] = -INFINITY;
                        const float top = largest(x) * fg;
                        if (__any_sync(kFullMask, top > M + 11.f)) move(top, g);
                        uint32_t y[16];
                        weigh_rounded(x, x, fg);
                        pack(x, y);
                        tmem_st16(scol + 16 * g, y);
                        if (own) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] *= vinv[info * TK + 32 * g + e];
                        }
                        add(x);
                    }
                }
                const float2 z = unpack2(add2(sum[0], sum[1]));
                l += z.x + z.y;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0 && arrives(2, p.count)) mbar_arrive(&pready[i]);
            }
            // ---- the rows' results
            ok = warp_wait(&odone, p.count & 1, &s_abort) && ok;  // the next piece's rows overwrite these, too
            if (slot < SLOTS) {
                tc_fence_after();
                float *other = reinterpret_cast<float *>(sk);  // the second O of a dual item: [D][128 rows]
                float f0 = 1.f, f1 = 0.f;
                if (p.dual) {
                    if (slot == 1 && busy) {
                        sml[r] = make_float2(M, mine ? l : 0.f);
#pragma unroll 1
                        for (int g = 0; g < D / 16 && mine; ++g) {
                            float x[16];
                            tmem_ld16(ocol + 16 * g, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) other[(16 * g + e) * 128 + r] = x[e];
                        }
                    }
                    named_barrier(1, 256);
                    const float2 y = sml[tr];
                    const float m = fmaxf(M, y.x);
                    f0 = ex2(M - m), f1 = p.nt > 1 ? ex2(y.x - m) : 0.f;
                    l = l * f0 + y.y * f1;
                    M = m;
                }
                // all lanes of a warp read tensor memory together
                const bool store = (!p.dual || slot == 0) && r < p.it.rows;
                // a broken wait must not pass for a result
                const float bad = ok && !*(volatile int *)&s_abort ? 1.f : NAN;
                const float norm = p.whole ? bad * (l > 0.f ? rsqrt_dim<D>() / l : 0.f) : bad;
                f0 *= norm, f1 *= norm;
                if ((!p.dual || slot == 0) && busy) {
                    auto row32 = [&](float (&x)[32], int col) {  // 32 columns, values in order
                        float y[32];
                        tmem_ld32(ocol + col, y);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            float z = (mine ? y[e] : 0.f) * f0;  // NaN where f0 is
                            if (p.dual && p.nt > 1) z = fmaf(other[(col + e) * 128 + r], f1, z);
                            x[(e & 24) + value_at(e & 7)] = z;
                        }
                    };
                    if (p.whole) {
                        // H of D = H of D / 32 over H of 32: 32 values of the result at a time
#pragma unroll 1
                        for (int q = 0; q < D / 32; ++q) {
                            float x[32];
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] = 0.f;
#pragma unroll 1
                            for (int j = 0; j < D / 32; ++j) {
                                const float sg = __popc(j & q) & 1 ? -1.f : 1.f;
                                float y[32];
                                row32(y, 32 * j);
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = fmaf(sg, y[e], x[e]);
                            }
#pragma unroll
                            for (int d = 1; d < 32; d <<= 1)
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(e & d)) {
                                        const float y = x[e], z = x[e + d];
                                        x[e] = y + z;
                                        x[e + d] = y - z;
                                    }
                            // by way of the query rows' place (their products are done): a lane
                            // has a row, and the stores want rows in one piece
#pragma unroll
                            for (int e = 0; e < 32; e += 8)
                                *reinterpret_cast<uint4 *>(sq + r * (D * 2) + (((q * 4 + e / 8) ^ (r & 7)) << 4)) =
                                    make_uint4(pack_bf16(x[e], x[e + 1]), pack_bf16(x[e + 2], x[e + 3]),
                                               pack_bf16(x[e + 4], x[e + 5]), pack_bf16(x[e + 6], x[e + 7]));
                        }
                        __syncwarp();
                        constexpr int CH = D / 8;  // 16-byte chunks of a row
                        const int base = r - lane, c = lane % CH;
#pragma unroll 1
                        for (int k = lane / CH; k < 32 && base + k < p.it.rows; k += 32 / CH) {
                            const int row = base + k, i = by_group(a, p.it.row0 + row);
                            const int h = p.hk * a.group + p.it.row0 + row - i * a.group;
                            *reinterpret_cast<uint4 *>(a.out + (p.s.t0 + i) * a.d.out_token_stride + (int64_t)h * D + c * 8) =
                                *reinterpret_cast<const uint4 *>(sq + row * (D * 2) + ((c ^ (row & 7)) << 4));
                        }
                    } else {
                        // planes of four values over the rows: the lanes' stores lie together
                        float4 *part = reinterpret_cast<float4 *>(parts + (int64_t)(blockIdx.x * 2 + slot_of(p)) * C::ROWS * C::PART) + r;
#pragma unroll 1
                        for (int g = 0; g < D / 32; ++g) {
                            float x[32];
                            row32(x, 32 * g);
                            if (store)
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    part[(8 * g + e / 4) * C::ROWS] = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
                        }
                        if (store) part[(D / 4) * C::ROWS] = make_float4(M, l, 0.f, 0.f);
                    }
                }
            }
            return true;
        });
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <int D, bool STALL>
cudaError_t launch(const RopeTable &tab, const AttnArgs &a, const AttnStall &stall, cudaStream_t st) {
    using C = Tiles<D>;
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_smem(k_attn_tiles<D, STALL>, C::SMEM, done);
    if (e != cudaSuccess) return e;
    const cudaError_t l = launch_early(k_attn_tiles<D, STALL>, dim3(kSms), kThreads, C::SMEM, st, tab, a, stall);
    return l != cudaSuccess ? l : launch_join<D, C::ROWS, true>(a, kSms, st);
}

}  // namespace

size_t attn_tiles_part_bytes(int head_dim) {
    const size_t rows = head_dim == 256 ? Tiles<256>::ROWS : Tiles<128>::ROWS;
    return 2 * rows * kSms * sizeof(float) * (head_dim + 4);
}

template <bool STALL>
static cudaError_t launch_any(const RopeTable &tab, const AttnArgs &a, const AttnStall &stall, cudaStream_t st) {
    if (a.c.head_dim == 64) return launch<64, STALL>(tab, a, stall, st);
    if (a.c.head_dim == 128) return launch<128, STALL>(tab, a, stall, st);
    return launch<256, STALL>(tab, a, stall, st);
}
cudaError_t launch_attn_tiles(const RopeTable &tab, const AttnArgs &a, cudaStream_t st) {
    return launch_any<false>(tab, a, AttnStall{}, st);
}
cudaError_t launch_attn_tiles_stalled(const RopeTable &tab, const AttnArgs &a, const AttnStall &stall, cudaStream_t st) {
    return launch_any<true>(tab, a, stall, st);
}

}  // namespace strata
