// rpa_rope.cu -- rotary positions and the write of new tokens into the paged cache.
//
// One launch takes q, k and v of a ragged batch (slices of a fused projection), rotates the rotary
// part of every q and k head by its token's position, writes q in its own type and K/V rows in the
// cache's type to the slots the page table names.
//
// The angle of pair i at position p is p w_i, w_i the double that rpa_rope_frequencies gives.  The handle
// keeps w_i / (2 pi) as a 64-bit binary fraction of a turn f_i, so that p f_i mod 2^64 is the angle's
// fraction of a turn in one integer product, exact but for f_i's own rounding (2^-65 of a turn a position, at
// most 2^-34 at 31 bits of position; 128-bit arithmetic makes f_i, for a quotient of doubles would be off by 2^-55.5
// a position).  The sine takes its upper 32 bits (2^-33 of a turn) as a float, whose 24 bits cost at most
// 2^-26 of a turn near half a turn, and nothing near 0.  In 32-bit floating point p w_i would be off by a
// tenth of a radian at a million positions, and in 64 bits the GPU runs it at 1/64 of the rate.
// Sines are computed once per token and pair, into shared memory, and serve all heads.
//
// A CTA takes a run of neighbouring tokens, up to 16 at a time, and looks their sequences, positions and slots up
// at once: cu_q_lens and kv_lens of up to 512 sequences go to shared memory whole (two dependent loads to the page
// id where a search in memory makes four: 8 k tokens 61.1 -> 60.1 us), beside more a warp searches a token's, 32
// probes at a time.  Then all threads compute the sines, and from there on
// there is only streaming: units of 16 elements (two 16-byte vectors of 2-byte types) of one row (q head, K
// row or V row).  A rotary unit is 8 pairs, both partners in one thread's registers (HALF: two vectors
// rotary_dim / 2 apart; INTERLEAVED: 16 neighbours), so that a row is read once and written once.  A thread
// keeps its place in the row and steps over the rows of all tokens, two rows' loads in flight; the first
// go out before the lookups.
//
// Bound by HBM: 8192 tokens of 64 q and 8 kv heads at D 128 (bf16, 344 MB) take 60 us, 5.7 TB/s, 0.84 of the
// measured copy.  Five CTAs an SM with two rows in flight a thread, when that took 61 us: four CTAs 63 us with two rows,
// 64 with four (spilled); one token a CTA 79 to 87 us.
//
// Rows of a 4-bit cache.  k is rotated in pairs of floats (sines by Taylor series, within 2^-30), k and v are divided by the cache's
// scales into pairs (within 2^-45), and a group's zero, scale and codes are rounded from the pairs' sums, so that they are those of the
// formula's real values but next to a border by as much (from 32-bit values some were others, most where a group lies far from zero).  A row's threads exchange it through shared memory, 16 neighbouring
// channels each, and form a group's extremes by shuffles.  Bound by instructions: 4.4 k tokens of 32 q and 8 kv heads at D 128 (groups
// of 32, 120 MB with the rows read back by the call behind) take 33 us, and the two calls 39 (one us of it for the lower halves in every code's sum).  One copy of the coding loop for q, K
// and V rows with the next row's loads in flight (57 -> 38 us then: unrolled by kind it did not stay in the instruction cache); three
// CTAs an SM of 12 tokens a round (80 registers; with four the loop spilled, 53 us); codes from the reciprocal of the
// scale, and the exact remainder only for those next to a border (no divisions).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include <cmath>
#include <new>

#include "rpa_internal.cuh"

using namespace rpa;

struct RpaRope {
    RpaRopeCfg cfg;
    int device, sms;
    unsigned long long* turns;  // device [rotary_dim / 2]: f_i
    int* status;                // device: first error since the last rpa_rope_get_status
};

namespace rpa {
namespace {

constexpr int kUnit = 16;       // elements of a unit
constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 5;    // resident an SM
constexpr int kRopeCtas4 = 3;   // ... that write a 4-bit cache
constexpr int kTokens = 16;     // tokens of a CTA's round
constexpr int kTokens4 = 12;    // ... that writes a 4-bit cache
constexpr int kSeqs = 512;      // sequences whose cu_q_lens and kv_lens a CTA reads into shared memory
constexpr int kMaxPairs = 288;  // rotary_dim <= 576

struct RopeParams {
    const uint8_t *q, *k, *v;
    size_t q_stride, k_stride, v_stride;  // bytes between tokens
    uint8_t *q_out, *kv;
    const int *kv_lens, *page_indices, *cu, *positions;
    const unsigned long long* turns;
    int* status;
    int S, T, Hq, Hkv, D, ps, P, N, latent;
    int rd, off;
    int rows;       // q heads + K rows + V rows of a token
    int per_row;    // units of a row
    int row_step;   // rows the CTA takes at once (its threads / per_row)
    int kt;         // KvType of the cache
    int group;      // channels of a group of a 4-bit cache
    int has_ks, has_vs;
    float magnitude, k_scale, v_scale;
};

template <typename T>
struct Vec8;  // eight elements as loaded
template <>
struct Vec8<float> {
    float4 a, b;
};
struct Half8 {
    uint4 a;
};
template <>
struct Vec8<__nv_bfloat16> : Half8 {};
template <>
struct Vec8<__half> : Half8 {};

__device__ __forceinline__ void load8(const uint8_t* p, Vec8<float>& v) {
    v.a = *reinterpret_cast<const float4*>(p);
    v.b = *reinterpret_cast<const float4*>(p + 16);
}
__device__ __forceinline__ void load8(const uint8_t* p, Half8& v) { v.a = *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void widen(const Vec8<float>& v, float* f) {
    f[0] = v.a.x; f[1] = v.a.y; f[2] = v.a.z; f[3] = v.a.w;
    f[4] = v.b.x; f[5] = v.b.y; f[6] = v.b.z; f[7] = v.b.w;
}
__device__ __forceinline__ void widen(const Vec8<__nv_bfloat16>& v, float* f) {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void widen(const Vec8<__half>& v, float* f) {
    const uint32_t w[4] = {v.a.x, v.a.y, v.a.z, v.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 h = f16x2_to_f32x2(w[i]);
        f[2 * i] = h.x;
        f[2 * i + 1] = h.y;
    }
}

template <bool F16>
__device__ __forceinline__ uint4 round8(const float* f) {
    return make_uint4(pack2<F16>(f[0], f[1]), pack2<F16>(f[2], f[3]), pack2<F16>(f[4], f[5]), pack2<F16>(f[6], f[7]));
}
__device__ __forceinline__ void store_q8(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store_q8(__nv_bfloat16* p, const float* f) { *reinterpret_cast<uint4*>(p) = round8<false>(f); }
__device__ __forceinline__ void store_q8(__half* p, const float* f) { *reinterpret_cast<uint4*>(p) = round8<true>(f); }

template <bool E5M2>
__device__ __forceinline__ uint32_t fp8x4(const float* f) {
    uint16_t lo, hi;
    if constexpr (E5M2) {
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
        asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
    } else {
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
    }
    return (uint32_t)lo | ((uint32_t)hi << 16);
}
__device__ __forceinline__ uint32_t int8x4(const float* f) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) r |= (uint32_t)(uint8_t)(int8_t)max(-128, min(127, __float2int_rn(f[i]))) << (8 * i);
    return r;
}
// Eight cache elements at element e of the row that starts at byte offset `row` of the cache.
__device__ __forceinline__ void store_kv8(uint8_t* kv, size_t row, int e, const float* f, int kt) {
    switch (kt) {
        case KT_BF16: *reinterpret_cast<uint4*>(kv + row + 2 * e) = round8<false>(f); break;
        case KT_F16: *reinterpret_cast<uint4*>(kv + row + 2 * e) = round8<true>(f); break;
        case KT_E4M3: *reinterpret_cast<uint2*>(kv + row + e) = make_uint2(fp8x4<false>(f), fp8x4<false>(f + 4)); break;
        case KT_E5M2: *reinterpret_cast<uint2*>(kv + row + e) = make_uint2(fp8x4<true>(f), fp8x4<true>(f + 4)); break;
        default: *reinterpret_cast<uint2*>(kv + row + e) = make_uint2(int8x4(f), int8x4(f + 4)); break;
    }
}

// least / greatest of three, NaN where any is
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float r;
    asm("min.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;\n" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The neighbour of a float16 value, below or above it
__device__ __forceinline__ __half next_half(__half x, bool up) {
    const unsigned short b = __half_as_ushort(x);
    if ((b & 0x7fff) == 0) return __ushort_as_half(up ? 0x0001 : 0x8001);
    return __ushort_as_half((unsigned short)(((b & 0x8000) != 0) == up ? b - 1 : b + 1));
}

// A pair of floats is their sum: `lo` holds what rounding `hi` left.  a + b as such a pair (any a, b; or |a| >= |b|).  (The intrinsics
// are not contracted: a product that a sum's rounding is measured against has to be rounded itself.)
__device__ __forceinline__ void two_sum(float a, float b, float& hi, float& lo) {
    const float h = __fadd_rn(a, b), c = __fsub_rn(h, a);
    lo = __fadd_rn(__fsub_rn(a, __fsub_rn(h, c)), __fsub_rn(b, c));
    hi = h;
}
__device__ __forceinline__ void quick_sum(float a, float b, float& hi, float& lo) {
    const float h = __fadd_rn(a, b);
    lo = __fsub_rn(b, __fsub_rn(h, a));
    hi = h;
}

// Cosine and sine of a fraction of a turn (in units of 2^-64) as pairs, off by 2^-30 at most: the Taylor series about the nearest
// quarter turn, their leading terms in pairs (the rest is below 2.6e-3, and 32 bits of it are enough).
__device__ __forceinline__ void sincos_pairs(unsigned long long turn, float2& cs, float2& sn) {
    const unsigned long long quarter = (turn + (1ull << 61)) >> 62;
    const long long r = (long long)(turn - (quarter << 62));  // up to an eighth of a turn
    const float fh = (float)(int)(r >> 32), fl = (float)(r - ((long long)(int)fh << 32));
    const float th = fh * 2.3283064365386963e-10f, tl = fl * 5.421010862427522e-20f;  // 2^-32, 2^-64
    constexpr float kPi = 6.2831854820251465f, kPiLo = -1.7484555314695172e-07f;      // 2 pi
    float xh = __fmul_rn(th, kPi), xl = fmaf(th, kPi, -xh) + (th * kPiLo + tl * kPi);
    quick_sum(xh, xl, xh, xl);
    const float sh = __fmul_rn(xh, xh), sl = fmaf(xh, xh, -sh) + 2.f * xh * xl;  // x^2
    // sine: x - x^3 / 6 + x^5 (1 / 120 - ...)
    {
        constexpr float kSixth = 0.1666666716337204f, kSixthLo = -4.967053879312289e-09f;
        const float ch = __fmul_rn(sh, xh), cl = fmaf(sh, xh, -ch) + (sh * xl + sl * xh);
        const float vh = __fmul_rn(ch, kSixth), vl = fmaf(ch, kSixth, -vh) + (ch * kSixthLo + cl * kSixth);
        const float rest = ch * sh * fmaf(sh, fmaf(sh, fmaf(sh, -2.50521084e-08f, 2.75573192e-06f), -1.98412698e-04f), 8.33333333e-03f);
        float h, l;
        quick_sum(xh, -vh, h, l);
        quick_sum(h, l + (rest + (xl - vl)), sn.x, sn.y);
    }
    // cosine: 1 - x^2 / 2 + x^4 / 24 - x^6 (1 / 720 - ...)
    {
        constexpr float k24 = 0.0416666679084301f, k24Lo = -1.2417634698280722e-09f;
        const float qh = __fmul_rn(sh, sh), ql = fmaf(sh, sh, -qh) + 2.f * sh * sl;
        const float gh = __fmul_rn(qh, k24), gl = fmaf(qh, k24, -gh) + (qh * k24Lo + ql * k24);
        const float rest = qh * sh * fmaf(sh, fmaf(sh, -2.75573192e-07f, 2.48015873e-05f), -1.38888889e-03f);
        float h, l, h2, l2;
        quick_sum(1.f, -0.5f * sh, h, l);
        quick_sum(h, gh, h2, l2);
        quick_sum(h2, (l2 + l) + (rest + (gl - 0.5f * sl)), cs.x, cs.y);
    }
    if (quarter & 1) {
        const float2 c = cs;
        cs = make_float2(-sn.x, -sn.y);
        sn = c;
    }
    if (quarter & 2) {
        cs = make_float2(-cs.x, -cs.y);
        sn = make_float2(-sn.x, -sn.y);
    }
}
// u c - w s of pairs c, s, as a pair
__device__ __forceinline__ void turn_pair(float u, float w, float ch, float cl, float sh, float sl, float& hi, float& lo) {
    const float p = __fmul_rn(u, ch), q = __fmul_rn(w, sh);
    float h, l;
    two_sum(p, -q, h, l);
    l += (fmaf(u, ch, -p) - fmaf(w, sh, -q)) + (u * cl - w * sl);
    quick_sum(h, fabsf(h) < INFINITY ? l : 0.f, hi, lo);
}

// A row of a 4-bit cache.  The row's D / 16 threads (neighbouring lanes, `mask`) hold its values by the pairs they turn, as sums
// y + yl; through `row` (shared, D floats) each takes 16 neighbouring channels, and a group's extremes come by shuffles.
// A group's zero and scale are rounded to one side, and its codes to the nearest: each step from the exact values of the sums, so
// that what 32 bits round away decides no code, and a group's codes do not hang on how its angles' sines were rounded.
__device__ __forceinline__ void store_int4(const RopeParams& p, const float* y, const float* yl, int e0, int e1, float* row, int place,
                                           uint32_t mask, long long slot, int h, bool is_v) {
    auto exchange = [&](const float* from, float* to) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            reinterpret_cast<float4*>(row + e0)[i] = make_float4(from[4 * i], from[4 * i + 1], from[4 * i + 2], from[4 * i + 3]);
            reinterpret_cast<float4*>(row + e1)[i] = make_float4(from[8 + 4 * i], from[9 + 4 * i], from[10 + 4 * i], from[11 + 4 * i]);
        }
        __syncwarp(mask);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(row + 16 * place)[i];
            to[4 * i] = v.x; to[4 * i + 1] = v.y; to[4 * i + 2] = v.z; to[4 * i + 3] = v.w;
        }
        __syncwarp(mask);  // the buffer is free again
    };
    float x[16], xl[16];
    exchange(y, x);
    const bool pairs = !is_v || p.has_vs;  // V as it came has no lower halves
    if (pairs) {
        exchange(yl, xl);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) xl[i] = 0.f;
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 16; i += 2) {
        lo = min_nan(lo, x[i], x[min(i + 1, 15)]);
        hi = max_nan(hi, x[i], x[min(i + 1, 15)]);
    }
    for (int o = 1; o < p.group / 16; o <<= 1) {
        const float l = __shfl_xor_sync(mask, lo, o), h2 = __shfl_xor_sync(mask, hi, o);
        lo = min_nan(lo, l, l);
        hi = max_nan(hi, h2, h2);
    }
    if (lo <= -65504.f || hi >= 65504.f) {  // (all of a group's threads)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (fabsf(x[i]) > 65504.f || (fabsf(x[i]) == 65504.f && x[i] * xl[i] > 0.f)) xl[i] = 0.f;
            x[i] = fminf(fmaxf(x[i], -65504.f), 65504.f);
        }
        lo = fminf(fmaxf(lo, -65504.f), 65504.f);
        hi = fminf(fmaxf(hi, -65504.f), 65504.f);
    }
    float lol = 0.f, hil = 0.f;  // what the extremes' own rounding left
    if (pairs) {
        lol = INFINITY;
        hil = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            lol = x[i] == lo ? fminf(lol, xl[i]) : lol;
            hil = x[i] == hi ? fmaxf(hil, xl[i]) : hil;
        }
        for (int o = 1; o < p.group / 16; o <<= 1) {
            lol = fminf(lol, __shfl_xor_sync(mask, lol, o));
            hil = fmaxf(hil, __shfl_xor_sync(mask, hil, o));
        }
    }
    __half zero = __float2half_rd(lo);
    if (__half2float(zero) == lo && lol < 0.f && lo > -65504.f) zero = next_half(zero, false);
    const float z = __half2float(zero);
    float dh, dl;
    two_sum(hi, -z, dh, dl);
    two_sum(dh, dl + hil, dh, dl);  // (far from zero a value's lower half is no small part of the group's range)
    __half scale = __float2half_ru(__fdiv_rn(dh, 15.f));
    {
        const float c = 15.f * __half2float(scale), b = 15.f * __half2float(next_half(scale, false));  // (exact)
        if (c < dh || (c == dh && dl > 0.f)) scale = next_half(scale, true);
        else if (b >= 0.f && (b > dh || (b == dh && dl <= 0.f))) scale = next_half(scale, false);
    }
    const float s = __half2float(scale), inv = __frcp_rn(s);
    // The quotient's nearest integer, to even: of (x - z + xl) (1 / s), off by less than 2^-17 for codes up to 15, unless one of the
    // thread's lies so near the middle of two that only the exact remainder says which.  (1.5 2^23 leaves a sum's integer in its low
    // bits, which are collected with their factors 16^i; what that constant's own bits add comes off at the end.)
    constexpr float kMagic = 12582912.f;
    constexpr uint32_t kBits = 0x4b400000u * 0x11111111u;
    uint32_t w[2] = {0, 0};
    float off = 0.f;
    const uint64_t nz2 = f32x2(-z, -z), inv2 = f32x2(inv, inv), magic2 = f32x2(kMagic, kMagic), back2 = f32x2(-kMagic, -kMagic);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
        const uint64_t t = fmul2(fadd2(fadd2(f32x2(x[i], x[i + 1]), nz2), f32x2(xl[i], xl[i + 1])), inv2), n = fadd2(t, magic2);
        float r0, r1, t0, t1, n0, n1;
        f32x2_split(fadd2(n, back2), r0, r1);
        f32x2_split(t, t0, t1);
        f32x2_split(n, n0, n1);
        off = max_nan(off, fabsf(t0 - r0), fabsf(t1 - r1));
        w[i / 8] += __float_as_uint(n0) * (1u << (4 * (i % 8))) + __float_as_uint(n1) * (1u << (4 * (i % 8) + 4));
    }
    w[0] -= kBits;
    w[1] -= kBits;
    if (!(off < 0.49999f)) {  // (also where the group has no range, or a NaN: 0 / 0 and NaN give 0)
        w[0] = w[1] = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // what r steps leave of the difference, exactly, against half a step
            float d, e;
            two_sum(x[i], -z, d, e);
            two_sum(d, e + xl[i], d, e);
            const float r = rintf(d * inv), left = fmaf(-r, s, d), up = (left - 0.5f * s) + e, down = (left + 0.5f * s) + e;
            int c = r == r ? (int)r : 0;
            const bool odd = c & 1;
            if (up > 0.f || (up == 0.f && odd)) ++c;
            if (down < 0.f || (down == 0.f && odd)) --c;
            w[i / 8] |= (uint32_t)min(max(c, 0), 15) << (4 * (i % 8));
        }
    }
    const int page = (int)(slot >> 32), at = (int)slot, ng = p.D / p.group;
    uint8_t* block = p.kv + ((size_t)page * p.Hkv + h) * ((size_t)p.ps * int4_key_bytes(p.D, p.group));
    uint8_t* codes = block + (size_t)((is_v ? p.ps : 0) + at) * (p.D / 2);
    *reinterpret_cast<uint2*>(codes + int4_chunk(place / 2, at, p.D) * 16 + (place & 1) * 8) = make_uint2(w[0], w[1]);
    if ((16 * place) % p.group == 0)
        reinterpret_cast<__half2*>(block + (size_t)p.ps * p.D)[(size_t)((is_v ? p.ps : 0) + at) * ng + 16 * place / p.group] =
            __halves2half2(scale, zero);
}

template <typename QT, bool HALF, bool INT4>
__global__ void __launch_bounds__(kRopeThreads, INT4 ? kRopeCtas4 : kRopeCtas) rpa_rope_kernel(const RopeParams p) {
    constexpr int kBatch = sizeof(QT) == 4 || INT4 ? 1 : 2;  // rows whose loads a thread has in flight (INT4: beside the one at work)
    constexpr int kRound = INT4 ? kTokens4 : kTokens;
    // [tokens][4][places] pairs of (cos, sin): place's pairs 2 i and 2 i + 1 at [i][place], so that neighbouring
    // places read neighbouring 16 bytes
    extern __shared__ float4 s_cs[];
    __shared__ long long s_slot[kRound];  // cache slot of a token (page * page_size + place; INT4: page, place), or -1
    __shared__ __align__(16) float s_rows[INT4 ? kRopeThreads * kUnit : 4];  // INT4: the rows that are being coded
    __shared__ int s_pos[kRound], s_live[kRound];
    __shared__ int s_cu[kSeqs + 1], s_kl[kSeqs];
    __shared__ unsigned long long s_turns[kMaxPairs];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int place = tid % p.per_row, row0 = tid / p.per_row;
    // this thread's unit: elements [e0, e0 + 8) and [e1, e1 + 8) of a row
    const int places = p.rd / kUnit;  // rotary units of a row
    const bool rot = place < places;
    int e0, e1;
    if (rot) {
        e0 = p.off + place * (HALF ? 8 : 16);
        e1 = e0 + (HALF ? p.rd / 2 : 8);
    } else {
        const int c = (place - places) * 16;  // of the elements outside the rotary part
        e0 = c < p.off ? c : c + p.rd;
        e1 = c + 8 < p.off ? c + 8 : c + 8 + p.rd;
    }
    const int t_end = (int)((long long)p.T * (blockIdx.x + 1) / gridDim.x);
    int t0 = (int)((long long)p.T * blockIdx.x / gridDim.x);
    auto source = [&](int t, int r) -> const uint8_t* {
        const uint8_t* base = r < p.Hq ? p.q + (size_t)t * p.q_stride : r < p.Hq + p.Hkv ? p.k + (size_t)t * p.k_stride : p.v + (size_t)t * p.v_stride;
        const int h = r < p.Hq ? r : r < p.Hq + p.Hkv ? r - p.Hq : r - p.Hq - p.Hkv;
        return base + (size_t)h * p.D * sizeof(QT);
    };
    // token i of a round: its sequence (< 0: none), where it starts and how many tokens and keys it has
    auto look_up = [&](int i, int t, int s, int q0, int ql, int kl) {
        int live = 0, pos = 0;
        long long slot = -1;
        if (s >= 0 && q0 >= 0 && kl <= p.P * p.ps && ql <= kl && q0 + ql <= p.T) {
            live = 1;
            const int j = kl - ql + (t - q0);
            const int pg = p.page_indices[(size_t)s * p.P + j / p.ps];
            pos = p.positions ? p.positions[t] : j;
            if ((unsigned)pg < (unsigned)p.N) slot = INT4 ? ((long long)pg << 32) | (j % p.ps) : (long long)pg * p.ps + j % p.ps;
            else set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
        }
        s_live[i] = live;
        s_pos[i] = pos;
        s_slot[i] = slot;
    };
    pdl_trigger();
    for (int i = tid; i < p.rd / 2; i += kRopeThreads) s_turns[i] = p.turns[i];  // the handle's own
    pdl_wait();
    const bool few = p.S <= kSeqs;
    if (few) {
        for (int i = tid; i < p.S; i += kRopeThreads) {
            s_cu[i] = p.cu[i];
            s_kl[i] = p.kv_lens[i];
        }
        if (tid == 0) s_cu[p.S] = p.cu[p.S];
    }
    for (; t0 < t_end; t0 += kRound) {
        const int n = min(kRound, t_end - t0);
        Vec8<QT> x0[kBatch], x1[kBatch];
        // rows from (token `tk` of the round, row r) on, row_step apart, through the tokens
        auto next = [&](int& tk, int& r) {
            r += p.row_step;
            while (r >= p.rows) {
                r -= p.rows;
                ++tk;
            }
        };
        auto fetch = [&](int tk, int r) {
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (tk < n) {
                    const uint8_t* s = source(t0 + tk, r);
                    load8(s + e0 * sizeof(QT), x0[b]);
                    load8(s + e1 * sizeof(QT), x1[b]);
                }
                next(tk, r);
            }
        };
        int tk = row0 < p.row_step ? row0 / p.rows : n, r = row0 % p.rows;  // (576: 252 threads have a place)
        fetch(tk, r);
        if (few) {
            __syncthreads();
            if (tid < n) {
                const int t = t0 + tid, s = last_start(s_cu, p.S, t);
                const bool in = p.S > 0 && s_cu[s] <= t && t < s_cu[s + 1];
                look_up(tid, t, in ? s : -1, in ? s_cu[s] : 0, in ? s_cu[s + 1] - s_cu[s] : 0, in ? s_kl[s] : 0);
            }
        } else {
            for (int i = warp; i < n; i += warps) {
                const int t = t0 + i, s = find_seq(p.cu, p.S, t, lane);
                if (lane == 0) look_up(i, t, s, s < 0 ? 0 : p.cu[s], s < 0 ? 0 : p.cu[s + 1] - p.cu[s], s < 0 ? 0 : p.kv_lens[s]);
            }
        }
        __syncthreads();
        float2* cs2 = reinterpret_cast<float2*>(s_cs);
        for (int i = tid; i < n * (p.rd / 2); i += blockDim.x) {
            const int k = i / (p.rd / 2), pair = i - k * (p.rd / 2);
            // the angle's fraction of a turn, its upper 32 bits as half turns in [-1, 1)
            const unsigned long long f = s_turns[pair] * (unsigned long long)(long long)s_pos[k];
            const int at = ((k * 4 + (pair & 7) / 2) * places + pair / 8) * 2 + (pair & 1);
            if constexpr (INT4) {
                // pairs, their low halves in a second table: the keys' codes want them
                float2 c, s;
                sincos_pairs(f, c, s);
                const float m = p.magnitude, ch = __fmul_rn(c.x, m), sh = __fmul_rn(s.x, m);
                cs2[at] = make_float2(ch, sh);
                cs2[kRound * 8 * places + at] = make_float2(fmaf(c.x, m, -ch) + c.y * m, fmaf(s.x, m, -sh) + s.y * m);
            } else {
                float sn, cs;
                sincospif((float)(int)((f + 0x80000000ull) >> 32) * 4.656612873077393e-10f, &sn, &cs);
                cs2[at] = make_float2(cs * p.magnitude, sn * p.magnitude);
            }
        }
        __syncthreads();
        // one row of a token
        auto process = [&](int tb, int rb, const Vec8<QT>& v0, const Vec8<QT>& v1) {
            if (!s_live[tb]) return;
            float y[16];
            widen(v0, y);
            widen(v1, y + 8);
            float yl[INT4 ? 16 : 1];
            if constexpr (INT4) {
                if (rb >= p.Hq) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) yl[i] = 0.f;
                }
                if (rot && rb >= p.Hq && rb < p.Hq + p.Hkv) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 cs = s_cs[(tb * 4 + i) * places + place], cl = s_cs[(kRound * 4 + tb * 4 + i) * places + place];
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int m = 2 * i + j, a = HALF ? m : 2 * m, c = HALF ? m + 8 : 2 * m + 1;
                            const float co = j ? cs.z : cs.x, si = j ? cs.w : cs.y, col = j ? cl.z : cl.x, sil = j ? cl.w : cl.y;
                            const float u = y[a], w = y[c];
                            turn_pair(u, w, co, col, si, sil, y[a], yl[a]);
                            turn_pair(w, -u, co, col, si, sil, y[c], yl[c]);
                        }
                    }
                }
            }
            if (rot && rb < p.Hq + (INT4 ? 0 : p.Hkv)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 cs = s_cs[(tb * 4 + i) * places + place];  // cos, sin of pairs 2 i and 2 i + 1
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int m = 2 * i + j, a = HALF ? m : 2 * m, c = HALF ? m + 8 : 2 * m + 1;
                        const float co = j ? cs.z : cs.x, si = j ? cs.w : cs.y, u = y[a], w = y[c];
                        y[a] = u * co - w * si;
                        y[c] = w * co + u * si;
                    }
                }
            }
            if (rb < p.Hq) {
                QT* o = reinterpret_cast<QT*>(p.q_out) + ((size_t)(t0 + tb) * p.Hq + rb) * p.D;
                store_q8(o + e0, y);
                store_q8(o + e1, y + 8);
            } else if (s_slot[tb] >= 0) {
                const bool is_v = rb >= p.Hq + p.Hkv;
                const int h = rb - p.Hq - (is_v ? p.Hkv : 0);
                if (is_v ? p.has_vs : p.has_ks) {
                    const float sc = is_v ? p.v_scale : p.k_scale;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float u = y[i], quotient = __fdiv_rn(u, sc);
                        if constexpr (INT4) {
                            // (what the quotient's rounding left is a value's lower half too)
                            const float rest = (fmaf(-quotient, sc, u) + yl[i]) * __frcp_rn(sc);
                            quick_sum(quotient, fabsf(quotient) < INFINITY && fabsf(rest) < INFINITY ? rest : 0.f, y[i], yl[i]);
                        } else {
                            y[i] = quotient;
                        }
                    }
                }
                if constexpr (INT4) {
                    const uint32_t mask = ((1u << p.per_row) - 1u) << (lane - place % 32);
                    store_int4(p, y, yl, e0, e1, s_rows + (size_t)(tid - place) * kUnit, place, mask, s_slot[tb], h, is_v);
                    return;
                }
                const int rows = p.latent ? p.Hkv : 2 * p.Hkv;
                const size_t row = ((size_t)s_slot[tb] * rows + (p.latent ? h : 2 * h + (is_v ? 1 : 0))) * p.D *
                                   (kt_8bit(p.kt) ? 1 : 2);
                store_kv8(p.kv, row, e0, y, p.kt);
                store_kv8(p.kv, row, e1, y + 8, p.kt);
            }
        };
        if constexpr (INT4) {
            // (one copy of the code that makes codes: two are more than the instruction cache takes)
#pragma unroll 1
            while (tk < n) {
                const Vec8<QT> v0 = x0[0], v1 = x1[0];
                const int tb = tk, rb = r;
                next(tk, r);
                if (tk < n) fetch(tk, r);
                process(tb, rb, v0, v1);
            }
        } else {
            while (tk < n) {
                int tb = tk, rb = r;
#pragma unroll
                for (int b = 0; b < kBatch; ++b) {
                    if (tb < n) process(tb, rb, x0[b], x1[b]);
                    next(tb, rb);
                }
                tk = tb;
                r = rb;
                if (tk < n) fetch(tk, r);
            }
        }
        __syncthreads();  // the round's tables are free again
    }
    // the lengths of every sequence, once
    if (blockIdx.x == 0) {
        for (int s = tid; s < p.S; s += blockDim.x) {
            const int q0 = p.cu[s], q1 = p.cu[s + 1], kl = p.kv_lens[s];
            if (q0 < 0 || q1 < q0 || kl < 0 || kl > p.P * p.ps || q1 - q0 > kl || q1 > p.T)
                set_status(p.status, RPA_ERR_BAD_LENGTHS);
        }
    }
}

template <typename QT>
cudaError_t launch_rope(const RopeParams& p, int half, int grid, int threads, cudaStream_t st) {
    // at most 36 KB (4-bit: 12 tokens, two tables, rotary_dim <= 256: 24 KB)
    const size_t smem = (size_t)(p.kt == KT_I4 ? 2 * kTokens4 : kTokens) * (p.rd / 2) * sizeof(float2);
    if (p.kt == KT_I4)
        return half ? launch_pdl(rpa_rope_kernel<QT, true, true>, grid, threads, smem, st, p)
                    : launch_pdl(rpa_rope_kernel<QT, false, true>, grid, threads, smem, st, p);
    return half ? launch_pdl(rpa_rope_kernel<QT, true, false>, grid, threads, smem, st, p)
                : launch_pdl(rpa_rope_kernel<QT, false, false>, grid, threads, smem, st, p);
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

void frequencies(const RpaRopeCfg& c, double* w) {
    const int n = (int)(c.rotary_dim / 2);
    const double rd = (double)c.rotary_dim;
    double base = c.base;
    if (c.scaling == RPA_ROPE_BASE) base *= std::pow(c.factor, (double)n / (n - 1));
    double a = 0, b = 0;
    if (c.scaling == RPA_ROPE_INDEX) {
        const double at_high = rd * std::log(c.trained_len / (c.high * kTwoPi)) / (2 * std::log(c.base));
        const double at_low = rd * std::log(c.trained_len / (c.low * kTwoPi)) / (2 * std::log(c.base));
        a = std::fmax(std::floor(at_high), 0.0);
        b = std::fmin(std::ceil(at_low), rd - 1);
    }
    for (int i = 0; i < n; ++i) {
        const double x = std::pow(base, -(double)i / n);
        double t = 1;
        if (c.scaling == RPA_ROPE_LINEAR) t = 0;
        if (c.scaling == RPA_ROPE_ROTATIONS)
            t = std::fmin(std::fmax((c.trained_len * x / kTwoPi - c.low) / (c.high - c.low), 0.0), 1.0);
        if (c.scaling == RPA_ROPE_INDEX) t = 1 - std::fmin(std::fmax((i - a) / std::fmax(b - a, 1e-3), 0.0), 1.0);
        w[i] = t < 1 ? x * t + x / c.factor * (1 - t) : x;  // (the factor of NONE is not checked: it may be 0)
    }
}

// w / (2 pi) in units of 2^-64, to the nearest, for 0 <= w <= 1.  With w = m 2^e, m of 53 bits, it is
// m c 2^(e - 66), c = 2^129 / pi; of the product m c (181 bits) all but the lowest 64 are kept.
unsigned long long turns_of(double w) {
    constexpr unsigned long long c1 = 0xa2f9836e4e441529ull, c0 = 0xfc2757d1f534ddc1ull;  // c = c1 2^64 + c0
    int e = 0;
    const unsigned long long m = (unsigned long long)std::ldexp(std::frexp(w, &e), 53);
    const unsigned __int128 p = (unsigned __int128)m * c1 + (((unsigned __int128)m * c0) >> 64);
    const int drop = 55 - e;
    return drop > 127 ? 0ull : (unsigned long long)((p + ((unsigned __int128)1 << (drop - 1))) >> drop);
}

}  // namespace
}  // namespace rpa

extern "C" {

void rpa_rope_cfg_init(RpaRopeCfg* cfg) {
    if (!cfg) return;
    RpaCfg cache = cfg->cache;
    rpa_cfg_init(&cache);
    memset(cfg, 0, sizeof *cfg);
    cfg->cache = cache;
    cfg->rotary_dim = cache.head_dim;
    cfg->base = 10000.0;
    cfg->factor = 1.0;
    cfg->low = 1.0;
    cfg->high = 4.0;
    cfg->magnitude = 1.0;
}

int rpa_rope_validate_cfg(const RpaRopeCfg* c) {
    if (!c) return RPA_ERR_INVALID_ARG;
    const int v = rpa_validate_cfg(&c->cache);
    if (v != RPA_OK) return v;
    if (c->pairing != RPA_ROPE_HALF && c->pairing != RPA_ROPE_INTERLEAVED) return RPA_ERR_INVALID_ARG;
    if (c->scaling < RPA_ROPE_NONE || c->scaling > RPA_ROPE_INDEX) return RPA_ERR_INVALID_ARG;
    if (c->reserved != 0) return RPA_ERR_INVALID_ARG;
    if (!(std::isfinite(c->base) && c->base > 1.0)) return RPA_ERR_INVALID_ARG;
    if (!std::isfinite(c->magnitude) || !std::isfinite((float)c->magnitude)) return RPA_ERR_INVALID_ARG;
    if (c->scaling != RPA_ROPE_NONE && !(std::isfinite(c->factor) && c->factor >= 1.0)) return RPA_ERR_INVALID_ARG;
    if (c->scaling == RPA_ROPE_ROTATIONS || c->scaling == RPA_ROPE_INDEX) {
        if (!(std::isfinite(c->trained_len) && c->trained_len > 0)) return RPA_ERR_INVALID_ARG;
        if (!(c->low > 0 && c->low < c->high && std::isfinite(c->high))) return RPA_ERR_INVALID_ARG;
    }
    if (c->rotary_dim < 1 || c->rotary_offset < 0 || c->rotary_dim > c->cache.head_dim ||
        c->rotary_offset > c->cache.head_dim - c->rotary_dim)
        return RPA_ERR_INVALID_ARG;
    // a unit is eight pairs, in 16-byte vectors
    if (c->rotary_dim % kUnit || c->rotary_offset % 8) return RPA_ERR_UNSUPPORTED;
    // zero scales have no quotient
    if ((c->cache.has_k_scale && c->cache.k_scale == 0.f) || (c->cache.has_v_scale && c->cache.v_scale == 0.f))
        return RPA_ERR_INVALID_ARG;
    return RPA_OK;
}

int rpa_rope_frequencies(const RpaRopeCfg* cfg, double* w) {
    if (!w) return RPA_ERR_INVALID_ARG;
    const int v = rpa_rope_validate_cfg(cfg);
    if (v == RPA_OK) frequencies(*cfg, w);
    return v;
}

int rpa_rope_create(const RpaRopeCfg* cfg, RpaRope** out) {
    if (!out) return RPA_ERR_INVALID_ARG;
    *out = nullptr;
    const int v = rpa_rope_validate_cfg(cfg);
    if (v != RPA_OK) return v;
    RpaRope* h = new (std::nothrow) RpaRope;
    if (!h) return RPA_ERR_CUDA;
    memset(h, 0, sizeof *h);
    h->cfg = *cfg;
    // f_i = w_i / (2 pi) in units of 2^-64 turns (w_i <= 1 rad, so f_i < 2^62)
    double w[kMaxPairs];
    unsigned long long f[kMaxPairs + 1] = {};  // the status word behind them starts at 0
    frequencies(*cfg, w);
    const int n = (int)(cfg->rotary_dim / 2);
    for (int i = 0; i < n; ++i) f[i] = turns_of(w[i]);
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess ||
        cudaMalloc(&h->turns, (size_t)(n + 1) * sizeof f[0]) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return RPA_ERR_CUDA;
    }
    if (!set_now(cudaMemcpy(h->turns, f, (size_t)(n + 1) * sizeof f[0], cudaMemcpyHostToDevice))) {
        cudaGetLastError();
        cudaFree(h->turns);
        delete h;
        return RPA_ERR_CUDA;
    }
    h->status = reinterpret_cast<int*>(h->turns + n);
    *out = h;
    return RPA_OK;
}

int rpa_rope_append(RpaRope* h, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                    int64_t v_stride, void* kv_pages, const int32_t* kv_lens, const int32_t* page_indices,
                    const int32_t* cu_q_lens, const int32_t* positions, int32_t num_seqs, void* q_out, void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    const RpaCfg& c = h->cfg.cache;
    const bool latent = c.kv_layout == RPA_KV_LATENT;
    const int64_t eb = c.q_dtype == RPA_DT_F32 ? 4 : 2;
    if (num_seqs < 0 || num_seqs > c.max_num_seqs) return RPA_ERR_INVALID_ARG;
    if (!kv_pages || !kv_lens || !page_indices || !cu_q_lens) return RPA_ERR_INVALID_ARG;
    if (latent ? v != nullptr : (c.num_q_tokens > 0 && !v)) return RPA_ERR_INVALID_ARG;
    if (c.num_q_tokens > 0 && (!q || !k || !q_out)) return RPA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(kv_pages, 16) ||
        !aligned(kv_lens, 4) || !aligned(page_indices, 4) || !aligned(cu_q_lens, 4) || !aligned(positions, 4))
        return RPA_ERR_INVALID_ARG;
    const int64_t strides[3] = {q_stride, k_stride, latent ? c.num_kv_heads * c.head_dim : v_stride};
    for (int i = 0; i < 3; ++i)
        if (strides[i] < (i ? c.num_kv_heads : c.num_q_heads) * c.head_dim || strides[i] % (16 / eb) ||
            strides[i] >= (int64_t)1 << 40)
            return RPA_ERR_INVALID_ARG;
    // in place a token's row of q is its row of q_out, or the rows of other tokens would be written over before they are read
    if (q_out == q && c.num_q_tokens > 1 && q_stride != c.num_q_heads * c.head_dim) return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok) return RPA_ERR_CUDA;
    RopeParams p;
    p.q = static_cast<const uint8_t*>(q);
    p.k = static_cast<const uint8_t*>(k);
    p.v = static_cast<const uint8_t*>(v);
    p.q_stride = (size_t)(strides[0] * eb);
    p.k_stride = (size_t)(strides[1] * eb);
    p.v_stride = (size_t)(strides[2] * eb);
    p.q_out = static_cast<uint8_t*>(q_out);
    p.kv = static_cast<uint8_t*>(kv_pages);
    p.kv_lens = kv_lens;
    p.page_indices = page_indices;
    p.cu = cu_q_lens;
    p.positions = positions;
    p.turns = h->turns;
    p.status = h->status;
    p.S = num_seqs;
    p.T = (int)c.num_q_tokens;
    p.Hq = (int)c.num_q_heads;
    p.Hkv = (int)c.num_kv_heads;
    p.D = (int)c.head_dim;
    p.ps = (int)c.page_size;
    p.P = (int)c.pages_per_seq;
    p.N = (int)c.total_num_pages;
    p.latent = latent;
    p.rd = (int)h->cfg.rotary_dim;
    p.off = (int)h->cfg.rotary_offset;
    p.rows = p.Hq + (latent ? 1 : 2) * p.Hkv;
    p.per_row = p.D / kUnit;
    p.row_step = kRopeThreads / p.per_row;
    p.kt = kv_type(c.kv_dtype);
    p.group = int4_group(c.kv_dtype);
    p.has_ks = c.has_k_scale;
    p.has_vs = c.has_v_scale;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.magnitude = (float)h->cfg.magnitude;
    const int threads = kRopeThreads, half = h->cfg.pairing == RPA_ROPE_HALF;
    // a token a CTA at least; without tokens one CTA still checks the lengths
    const int most = h->sms * (p.kt == KT_I4 ? kRopeCtas4 : kRopeCtas), grid = p.T < 1 ? 1 : p.T < most ? p.T : most;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = c.q_dtype == RPA_DT_F32   ? launch_rope<float>(p, half, grid, threads, st)
                          : c.q_dtype == RPA_DT_F16 ? launch_rope<__half>(p, half, grid, threads, st)
                                                    : launch_rope<__nv_bfloat16>(p, half, grid, threads, st);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return RPA_ERR_CUDA;
    }
    return RPA_OK;
}

int rpa_rope_read(RpaRope* h, const void* kv_pages, const int32_t* kv_lens, const int32_t* page_indices,
                  const int32_t* cu_q_lens, int32_t num_seqs, void* k_out, void* v_out, void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    const RpaCfg& c = h->cfg.cache;
    const bool latent = c.kv_layout == RPA_KV_LATENT;
    if (num_seqs < 0 || num_seqs > c.max_num_seqs) return RPA_ERR_INVALID_ARG;
    if (!kv_pages || !kv_lens || !page_indices || !cu_q_lens) return RPA_ERR_INVALID_ARG;
    if (c.num_q_tokens > 0 && (!k_out || (!latent && !v_out))) return RPA_ERR_INVALID_ARG;
    if (latent && v_out) return RPA_ERR_INVALID_ARG;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(kv_pages, 16) || !aligned(kv_lens, 4) ||
        !aligned(page_indices, 4) || !aligned(cu_q_lens, 4))
        return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok) return RPA_ERR_CUDA;
    ReadParams p;
    p.kv = static_cast<const uint8_t*>(kv_pages);
    p.k = static_cast<uint8_t*>(k_out);
    p.v = static_cast<uint8_t*>(v_out);
    p.kv_lens = kv_lens;
    p.page_indices = page_indices;
    p.cu = cu_q_lens;
    p.status = h->status;
    p.S = num_seqs;
    p.T = (int)c.num_q_tokens;
    p.Hkv = (int)c.num_kv_heads;
    p.D = (int)c.head_dim;
    p.ps = (int)c.page_size;
    p.P = (int)c.pages_per_seq;
    p.N = (int)c.total_num_pages;
    p.latent = latent;
    p.kt = kv_type(c.kv_dtype);
    p.group = int4_group(c.kv_dtype);
    p.k_scale = c.has_k_scale ? c.k_scale : 1.f;
    p.v_scale = c.has_v_scale ? c.v_scale : 1.f;
    p.wide = aligned(k_out, 32) && aligned(v_out, 32);
    if (launch_read(p, c.q_dtype, h->sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return RPA_ERR_CUDA;
    }
    return RPA_OK;
}

int rpa_rope_get_status(RpaRope* h, void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    return g.ok ? take_status(h->status, static_cast<cudaStream_t>(stream)) : RPA_ERR_CUDA;
}

void rpa_rope_destroy(RpaRope* h) {
    if (!h) return;
    DeviceGuard g(h->device);
    cudaFree(h->turns);
    delete h;
}

}  // extern "C"
