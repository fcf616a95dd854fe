// rpa_read.cu -- rows of the paged cache as values (rpa_rope_read).
//
// Token t of a ragged batch stands for one slot of its sequence, as in the append; its K and V rows come out as
// values of q's type: a 2- or 1-byte element times the cache's scale, or code * scale + zero of a 4-bit group
// (the product of a 4-bit code and an 11-bit scale is exact in 32 bits, so the sum rounds once), times the cache's scale.
//
// A CTA takes blocks of neighbouring tokens (as many as its threads hold a row's units of 16 elements of: 32 at D 128), looks
// their slots up at once, and then a thread steps over the rows of its token, four in flight.  Neighbouring threads hold a row's
// units, then the same row of the next token: in a 4-bit block the rows of neighbouring slots lie side by side.  Few tokens spread
// over CTAs by rows.  Bound by HBM, the rows read and written: 53.5 k tokens of 8 kv heads at D 128 (groups of 128, 278 MB) take 48 us,
// 5.8 TB/s, 52 in a stream of calls; 1300 tokens 5.3 us and a call 6, of launch, lookups and two dependent loads.  A row of every
// token a thread, not every row of a token a warp (75 -> 57 us), and codes two at a time (57 -> 52).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "rpa_internal.cuh"

namespace rpa {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadCtas = 4;     // resident an SM
constexpr int kReadSeqs = 512;    // sequences whose cu_q_lens and kv_lens a CTA reads into shared memory
constexpr int kReadFly = 4;      // rows whose loads a thread has in flight

enum ReadMode : int { kRead16 = 0, kRead8 = 1, kRead4 = 2 };

template <int MODE>
struct Unit16 {  // 16 elements as loaded
    uint4 a[MODE == kRead16 ? 2 : 1];
};
template <>
struct Unit16<kRead4> {
    uint2 codes;
    uint32_t scale_zero;
};

// Sixteen elements; where the output starts on 32 bytes (`wide`) a sector in one store.
__device__ __forceinline__ void put_words(void* o, const uint32_t* w, int n, bool wide) {
#pragma unroll
    for (int i = 0; i < n; i += 8) {
        if (wide) {
            store_32(static_cast<uint32_t*>(o) + i, w + i);
        } else {
            static_cast<uint4*>(o)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
            static_cast<uint4*>(o)[i / 4 + 1] = make_uint4(w[i + 4], w[i + 5], w[i + 6], w[i + 7]);
        }
    }
}
__device__ __forceinline__ void put16(float* o, const float* f, bool wide) {
    uint32_t w[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(f[i]);
    put_words(o, w, 16, wide);
}
template <bool F16>
__device__ __forceinline__ void put16_2(void* o, const float* f, bool wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<F16>(f[2 * i], f[2 * i + 1]);
    put_words(o, w, 8, wide);
}
__device__ __forceinline__ void put16(__nv_bfloat16* o, const float* f, bool wide) { put16_2<false>(o, f, wide); }
__device__ __forceinline__ void put16(__half* o, const float* f, bool wide) { put16_2<true>(o, f, wide); }

// Where a token's rows lie: its unit of K of kv head 0, from there on a head's and V's, and of a 4-bit cache the same of the pairs.
template <int MODE>
struct Rows {
    const uint8_t *at, *pair;
    uint32_t head, v, pair_v;
    __device__ __forceinline__ Rows(const ReadParams& p, int page, int slot, int place) {
        if constexpr (MODE == kRead4) {
            const int ng = p.D / p.group;
            head = (uint32_t)(p.ps * int4_key_bytes(p.D, p.group));
            const uint8_t* block = p.kv + (size_t)page * p.Hkv * head;
            at = block + (uint32_t)(slot * (p.D / 2) + int4_chunk(place / 2, slot, p.D) * 16 + (place & 1) * 8);
            pair = block + (uint32_t)(p.ps * p.D + slot * ng * 4 + 16 * place / p.group * 4);
            v = (uint32_t)(p.ps * (p.D / 2));
            pair_v = (uint32_t)(p.ps * ng * 4);
        } else {
            const uint32_t row = (uint32_t)p.D * (MODE == kRead16 ? 2 : 1);
            head = p.latent ? row : 2 * row;
            at = p.kv + ((size_t)page * p.ps + slot) * ((size_t)p.Hkv * head) + 16 * place * (MODE == kRead16 ? 2 : 1);
            v = row;
        }
    }
    __device__ __forceinline__ void load(int h, bool is_v, Unit16<MODE>& x) const {
        const uint8_t* s = at + (size_t)h * head + (is_v ? v : 0u);
        if constexpr (MODE == kRead4) {
            x.codes = *reinterpret_cast<const uint2*>(s);
            x.scale_zero = *reinterpret_cast<const uint32_t*>(pair + (size_t)h * head + (is_v ? pair_v : 0u));
        } else {
#pragma unroll
            for (int k = 0; k < (MODE == kRead16 ? 2 : 1); ++k) x.a[k] = reinterpret_cast<const uint4*>(s)[k];
        }
    }
};
template <int MODE>
__device__ __forceinline__ void widen(const Unit16<MODE>& x, int kt, float* f) {
    if constexpr (MODE == kRead4) {
        int4_values(x.codes, f16x2_to_f32x2(x.scale_zero), f);
    } else if constexpr (MODE == kRead16) {
        const uint32_t w[8] = {x.a[0].x, x.a[0].y, x.a[0].z, x.a[0].w, x.a[1].x, x.a[1].y, x.a[1].z, x.a[1].w};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 v = kt == KT_F16 ? f16x2_to_f32x2(w[k]) : make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
            f[2 * k] = v.x;
            f[2 * k + 1] = v.y;
        }
    } else {
        const uint32_t w[4] = {x.a[0].x, x.a[0].y, x.a[0].z, x.a[0].w};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 v = kt == KT_I8     ? cvt8x8_to_f16x8<KT_I8>(w[2 * k], w[2 * k + 1])
                            : kt == KT_E5M2 ? cvt8x8_to_f16x8<KT_E5M2>(w[2 * k], w[2 * k + 1])
                                            : cvt8x8_to_f16x8<KT_E4M3>(w[2 * k], w[2 * k + 1]);
            const uint32_t hv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                const float2 d = f16x2_to_f32x2(hv[m]);
                f[8 * k + 2 * m] = d.x;
                f[8 * k + 2 * m + 1] = d.y;
            }
        }
    }
}

template <typename QT, int MODE>
__global__ void __launch_bounds__(kReadThreads, kReadCtas) rpa_read_kernel(const ReadParams p) {
    __shared__ long long s_page[kReadThreads / 4];  // page and place of a token's slot (page << 32 | place), or -1
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_row = p.D / 16, rows = (p.latent ? 1 : 2) * p.Hkv;
    const int step = kReadThreads / per_row, place = tid % per_row, mine = tid / per_row;  // a thread: one unit of one token's rows
    const int blocks = (p.T + step - 1) / step;
    __shared__ int s_cu[kReadSeqs + 1], s_kl[kReadSeqs];
    pdl_trigger();
    pdl_wait();
    const bool few = p.S <= kReadSeqs;
    if (few) {
        for (int i = tid; i < p.S; i += kReadThreads) {
            s_cu[i] = p.cu[i];
            s_kl[i] = p.kv_lens[i];
        }
        if (tid == 0) s_cu[p.S] = p.cu[p.S];
        __syncthreads();
    }
    const long long tasks = (long long)blocks * rows;  // (block of tokens, row)
    long long task = tasks * blockIdx.x / gridDim.x;
    const long long end = tasks * (blockIdx.x + 1) / gridDim.x;
    while (task < end) {
        const int block = (int)(task / rows), r0 = (int)(task - (long long)block * rows);
        const int r1 = (int)min((long long)rows, r0 + (end - task));
        const int t0 = block * step, n = min(step, p.T - t0);
        // token i: its sequence (< 0: none), where that starts and how many tokens and keys it has
        auto look_up = [&](int i, int t, int s, int q0, int ql, int kl) {
            long long at = -1;
            if (s >= 0 && q0 >= 0 && kl <= p.P * p.ps && ql <= kl && q0 + ql <= p.T) {
                const int j = kl - ql + (t - q0), pg = p.page_indices[(size_t)s * p.P + j / p.ps];
                if ((unsigned)pg < (unsigned)p.N) at = ((long long)pg << 32) | (j % p.ps);
                else set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
            }
            s_page[i] = at;
        };
        if (few) {
            if (tid < n) {
                const int t = t0 + tid, s = last_start(s_cu, p.S, t);
                const bool in = p.S > 0 && s_cu[s] <= t && t < s_cu[s + 1];
                look_up(tid, t, in ? s : -1, in ? s_cu[s] : 0, in ? s_cu[s + 1] - s_cu[s] : 0, in ? s_kl[s] : 0);
            }
        } else {
            for (int i = warp; i < n; i += kReadThreads / 32) {
                const int t = t0 + i, s = find_seq(p.cu, p.S, t, lane);
                if (lane == 0) look_up(i, t, s, s < 0 ? 0 : p.cu[s], s < 0 ? 0 : p.cu[s + 1] - p.cu[s], s < 0 ? 0 : p.kv_lens[s]);
            }
        }
        __syncthreads();
        const long long slot = mine < n ? s_page[mine] : -1;
        if (slot >= 0) {
            const Rows<MODE> from(p, (int)(slot >> 32), (int)slot, place);
            const size_t out = ((size_t)(t0 + mine) * p.Hkv) * p.D + 16 * place;
            for (int r = r0; r < r1; r += kReadFly) {
                Unit16<MODE> x[kReadFly];
#pragma unroll
                for (int b = 0; b < kReadFly; ++b)
                    if (r + b < r1) from.load(r + b < p.Hkv ? r + b : r + b - p.Hkv, r + b >= p.Hkv, x[b]);
#pragma unroll
                for (int b = 0; b < kReadFly; ++b) {
                    if (r + b >= r1) break;
                    const bool is_v = r + b >= p.Hkv;
                    float f[16];
                    widen<MODE>(x[b], p.kt, f);
                    if constexpr (MODE == kRead4 && std::is_same<QT, __half>::value) int4_saturate(f16x2_to_f32x2(x[b].scale_zero), f);
                    const float sc = is_v ? p.v_scale : p.k_scale;
                    if (sc != 1.f) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) f[k] *= sc;
                    }
                    put16(reinterpret_cast<QT*>(is_v ? p.v : p.k) + out + (size_t)(is_v ? r + b - p.Hkv : r + b) * p.D, f, p.wide);
                }
            }
        }
        __syncthreads();  // the slots are looked up anew
        task += r1 - r0;
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
cudaError_t launch_as(const ReadParams& p, int grid, cudaStream_t st) {
    return p.kt == KT_I4      ? launch_pdl(rpa_read_kernel<QT, kRead4>, grid, kReadThreads, 0, st, p)
           : kt_8bit(p.kt) ? launch_pdl(rpa_read_kernel<QT, kRead8>, grid, kReadThreads, 0, st, p)
                              : launch_pdl(rpa_read_kernel<QT, kRead16>, grid, kReadThreads, 0, st, p);
}

}  // namespace

cudaError_t launch_read(const ReadParams& p, int q_dtype, int sms, cudaStream_t st) {
    // a (block of tokens, row) a CTA at least; without tokens one CTA still checks the lengths
    const int step = kReadThreads / (p.D / 16);
    const long long tasks = (long long)((p.T + step - 1) / step) * (p.latent ? 1 : 2) * p.Hkv, most = (long long)sms * kReadCtas;
    const int grid = (int)(tasks < 1 ? 1 : tasks < most ? tasks : most);
    return q_dtype == RPA_DT_F32   ? launch_as<float>(p, grid, st)
           : q_dtype == RPA_DT_F16 ? launch_as<__half>(p, grid, st)
                                   : launch_as<__nv_bfloat16>(p, grid, st);
}

}  // namespace rpa
