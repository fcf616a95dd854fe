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
constexpr int kTokens = 16;     // tokens of a CTA's round
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

template <typename QT, bool HALF>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rpa_rope_kernel(const RopeParams p) {
    constexpr int kBatch = sizeof(QT) == 4 ? 1 : 2;  // rows whose loads a thread has in flight
    // [tokens][4][places] pairs of (cos, sin): place's pairs 2 i and 2 i + 1 at [i][place], so that neighbouring
    // places read neighbouring 16 bytes
    extern __shared__ float4 s_cs[];
    __shared__ long long s_slot[kTokens];  // cache slot of a token (page * page_size + place), or -1
    __shared__ int s_pos[kTokens], s_live[kTokens];
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
            if ((unsigned)pg < (unsigned)p.N) slot = (long long)pg * p.ps + j % p.ps;
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
    for (; t0 < t_end; t0 += kTokens) {
        const int n = min(kTokens, t_end - t0);
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
                // the last sequence that starts at or before the token
                const int t = t0 + tid;
                int s = 0, end = p.S;
                while (end - s > 1) {
                    const int m = (s + end) / 2;
                    if (s_cu[m] <= t) s = m;
                    else end = m;
                }
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
            float sn, cs;
            sincospif((float)(int)((f + 0x80000000ull) >> 32) * 4.656612873077393e-10f, &sn, &cs);
            cs2[((k * 4 + (pair & 7) / 2) * places + pair / 8) * 2 + (pair & 1)] = make_float2(cs * p.magnitude, sn * p.magnitude);
        }
        __syncthreads();
        while (tk < n) {
            int tb = tk, rb = r;
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                if (tb < n && s_live[tb]) {
                    float y[16];
                    widen(x0[b], y);
                    widen(x1[b], y + 8);
                    if (rot && rb < p.Hq + p.Hkv) {
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
                            for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(y[i], sc);
                        }
                        const int rows = p.latent ? p.Hkv : 2 * p.Hkv;
                        const size_t row = ((size_t)s_slot[tb] * rows + (p.latent ? h : 2 * h + (is_v ? 1 : 0))) * p.D *
                                           (kt_8bit(p.kt) ? 1 : 2);
                        store_kv8(p.kv, row, e0, y, p.kt);
                        store_kv8(p.kv, row, e1, y + 8, p.kt);
                    }
                }
                next(tb, rb);
            }
            tk = tb;
            r = rb;
            if (tk < n) fetch(tk, r);
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
    const size_t smem = (size_t)kTokens * (p.rd / 2) * sizeof(float2);  // at most 36 KB
    return half ? launch_pdl(rpa_rope_kernel<QT, true>, grid, threads, smem, st, p)
                : launch_pdl(rpa_rope_kernel<QT, false>, grid, threads, smem, st, p);
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
    p.kt = c.kv_dtype == RPA_DT_F16 ? KT_F16 : c.kv_dtype == RPA_DT_FP8_E4M3 ? KT_E4M3
         : c.kv_dtype == RPA_DT_FP8_E5M2 ? KT_E5M2 : c.kv_dtype == RPA_DT_INT8 ? KT_I8 : KT_BF16;
    p.has_ks = c.has_k_scale;
    p.has_vs = c.has_v_scale;
    p.k_scale = c.k_scale;
    p.v_scale = c.v_scale;
    p.magnitude = (float)h->cfg.magnitude;
    const int threads = kRopeThreads, half = h->cfg.pairing == RPA_ROPE_HALF;
    // a token a CTA at least; without tokens one CTA still checks the lengths
    const int most = h->sms * kRopeCtas, grid = p.T < 1 ? 1 : p.T < most ? p.T : most;
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
