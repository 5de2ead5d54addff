// kv4_row.cuh -- device pieces shared by the kernels around the paged 4-bit
// cache (include/strata_attn.h): the rotary table, the Walsh-Hadamard
// transform of a row and the block rule of the codec (include/strata_kv.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/strata_attn.h"

// Frequencies of a rotary handle, passed to kernels by value: freq[i] is
// f_i / (2 pi) in turns per position, as a 64-bit fixed-point fraction.
struct RopeTable {
    uint64_t freq[STRATA_ROPE_MAX_HEAD_DIM / 2];
    double m;    // factor of cosine and sine
    int rd;      // rotary_dim; 0: no rotation
    int half;    // 1: pairs (i, i + rd/2), 0: pairs (2i, 2i + 1)
};

struct strata_rope_s {
    strata_rope_desc desc;
    RopeTable table;
};

// Check a cache description; on failure the reason is the last error.
strata_status strata_check_kv4_cache(const strata_kv4_cache *cache);

namespace strata {

constexpr unsigned kFullMask = 0xffffffffu;

// Frequency of pair i. The table is a kernel parameter; lanes ask for different
// entries, which the constant cache serves one at a time (32 replays a warp), so
// it is read through a pointer whose origin the compiler does not see, as memory.
__device__ __forceinline__ uint64_t rope_freq(const RopeTable &t, int i) {
    const uint64_t *p = t.freq;
    asm("" : "+l"(p));
    return p[i];
}

// position * f / (2 pi) modulo one turn: the product wraps modulo 2^64, which
// is exactly one turn, so a far position loses no bits. Unsigned, since only
// there wrapping is defined; read as a signed number it is the fraction of a
// half turn in [-1, 1).
__host__ __device__ __forceinline__ uint64_t turn_of(uint64_t freq, int32_t position) {
    return (uint64_t)(int64_t)position * freq;
}
__device__ __forceinline__ double half_turns(const RopeTable &t, int i, int position) {
    return (double)(int64_t)turn_of(rope_freq(t, i), position) * 0x1p-63;
}

// (cos, sin) of pair i: fp64, rounded once to fp32 (the bits that
// strata_rope_apply and strata_kv4_append promise)
__device__ __forceinline__ float2 rope_cs(const RopeTable &t, int i, int position) {
    double s, c;
    sincospi(half_turns(t, i, position), &s, &c);
    return make_float2((float)(c * t.m), (float)(s * t.m));
}

// the same in fp32, for a result that is not rounded to fixed bits: 32 bits of
// the turn's fraction, then the hardware's sine and cosine (off by 2^-20.9 at
// most in [-pi, pi]; the row is rounded to fp16, 2^-11, next)
__device__ __forceinline__ float2 rope_cs_f32(const RopeTable &t, int i, int position) {
    const int32_t turn = (int32_t)(turn_of(rope_freq(t, i), position) >> 32);
    const float x = (float)turn * 0x1.921fb6p-30f;  // pi 2^-31 a unit
    return make_float2(__cosf(x) * (float)t.m, __sinf(x) * (float)t.m);
}

// u c - v s and v c + u s, each product and each sum rounded once
__device__ __forceinline__ float rope_first(float u, float v, float2 cs) {
    return __fsub_rn(__fmul_rn(u, cs.x), __fmul_rn(v, cs.y));
}
__device__ __forceinline__ float rope_second(float u, float v, float2 cs) {
    return __fadd_rn(__fmul_rn(v, cs.x), __fmul_rn(u, cs.y));
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Rotary partner of value i < rd of a row, and its pair
__device__ __forceinline__ int rope_partner(const RopeTable &t, int i) {
    return t.half ? (i < t.rd / 2 ? i + t.rd / 2 : i - t.rd / 2) : (i ^ 1);
}
__device__ __forceinline__ int rope_pair(const RopeTable &t, int i) {
    return t.half ? (i < t.rd / 2 ? i : i - t.rd / 2) : (i >> 1);
}
__device__ __forceinline__ bool rope_is_second(const RopeTable &t, int i) {
    return t.half ? i >= t.rd / 2 : (i & 1) != 0;
}

// fp32(1 / sqrt(D)), the transform's normalisation
template <int D>
__device__ __forceinline__ float rsqrt_dim() {
    return D == 64 ? 0.125f : D == 128 ? 0.08838834764831844055f : 0.0625f;
}

// Unnormalised Walsh-Hadamard transform of a row held by a whole warp: lane l
// has values l * (D/32) .. + D/32 - 1. Used where the rounding order is free.
template <int D>
__device__ __forceinline__ void fwht_warp(float (&v)[D / 32], int lane) {
    constexpr int P = D / 32;
#pragma unroll
    for (int s = 1; s < P; s <<= 1)
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (!(i & s)) {
                const float a = v[i], b = v[i + s];
                v[i] = a + b;
                v[i + s] = a - b;
            }
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
        const float sg = (lane & s) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = fmaf(sg, v[i], __shfl_xor_sync(kFullMask, v[i], s));
    }
}

// One query row for the attention, held by a warp as fwht_warp lays it out, in
// three steps: the cosines and sines of a token (which its heads share), the
// loads, and rotary in fp32 with H x / sqrt(D) * scale.
template <int D>
struct QueryRow {
    static constexpr int P = D / 32;
    // value i -> x_i c_i + x_partner s_i
    static __device__ __forceinline__ void angles(float2 (&cs)[P], const RopeTable &t, int position, int lane) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const int i = lane * P + j;
            cs[j] = make_float2(1.f, 0.f);
            if (i < t.rd) {
                if (!t.half && (j & 1)) {
                    cs[j] = make_float2(cs[j - 1].x, -cs[j - 1].y);
                } else {
                    cs[j] = rope_cs_f32(t, rope_pair(t, i), position);
                    if (!rope_is_second(t, i)) cs[j].y = -cs[j].y;
                }
            }
        }
    }
    // the lane's values, and their partners in the half layout
    struct Raw {
        uint32_t x[P / 2], y[P / 2];
    };
    static __device__ __forceinline__ void words(uint32_t (&w)[P / 2], const __nv_bfloat16 *x) {
        if constexpr (P == 2) w[0] = *reinterpret_cast<const uint32_t *>(x);
        if constexpr (P == 4) *reinterpret_cast<uint2 *>(w) = *reinterpret_cast<const uint2 *>(x);
        if constexpr (P == 8) *reinterpret_cast<uint4 *>(w) = *reinterpret_cast<const uint4 *>(x);
    }
    static __device__ __forceinline__ void load(Raw &r, const __nv_bfloat16 *x, const RopeTable &t, int lane) {
        const int i = lane * P;
        words(r.x, x + i);
#pragma unroll
        for (int j = 0; j < P / 2; ++j) r.y[j] = 0u;
        if (!t.half || i >= t.rd) return;
        if (t.rd % (2 * P) == 0) {  // the partners of a lane lie together
            words(r.y, x + rope_partner(t, i));
        } else {
#pragma unroll
            for (int j = 0; j < P; ++j)
                if (i + j < t.rd)
                    r.y[j / 2] |= (uint32_t)__bfloat16_as_ushort(x[rope_partner(t, i + j)]) << (16 * (j & 1));
        }
    }
    static __device__ __forceinline__ void rotate(float (&v)[P], const Raw &r, const float2 (&cs)[P], const RopeTable &t,
                                                  int lane) {
        float x[P];
#pragma unroll
        for (int j = 0; j < P; ++j) x[j] = (j & 1) ? bf16_hi(r.x[j / 2]) : bf16_lo(r.x[j / 2]);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            const float y = t.half ? ((j & 1) ? bf16_hi(r.y[j / 2]) : bf16_lo(r.y[j / 2])) : x[j ^ 1];
            v[j] = lane * P + j < t.rd ? fmaf(y, cs[j].y, x[j] * cs[j].x) : x[j];
        }
    }
    static __device__ __forceinline__ void turn(float (&v)[P], const Raw &r, const float2 (&cs)[P], const RopeTable &t,
                                                float scale, int lane) {
        rotate(v, r, cs, t, lane);
        fwht_warp<D>(v, lane);
#pragma unroll
        for (int j = 0; j < P; ++j) v[j] *= rsqrt_dim<D>() * scale;
    }
};

}  // namespace strata
