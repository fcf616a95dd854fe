// rpa_read.cu -- rows of the paged cache as values (rpa_rope_read).
//
// Token t of a ragged batch stands for one slot of its sequence, as in the append; its K and V rows come out as
// values of q's type: a 2- or 1-byte element times the cache's scale, or code * scale + zero of a 4-bit group
// (the product of a 4-bit code and an 11-bit scale is exact in 32 bits, so the sum rounds once), times the cache's scale.
//
// A CTA takes a run of neighbouring tokens, up to 32 at a time, looks their slots up at once, and streams units of
// 16 elements of one row: neighbouring threads take a row's units, then the same row of the next token (in a
// 4-bit block the rows of neighbouring slots lie side by side), then the next row.  Bound by HBM: the rows read and written.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "rpa_internal.cuh"

namespace rpa {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadCtas = 4;     // resident an SM
constexpr int kReadTokens = 32;  // tokens of a CTA's round
constexpr int kReadFly = 4;      // units whose loads a thread has in flight

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

__device__ __forceinline__ void put16(float* o, const float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(o)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
template <bool F16>
__device__ __forceinline__ void put16_2(void* o, const float* f) {
    uint4* d = static_cast<uint4*>(o);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        d[i] = make_uint4(pack2<F16>(f[8 * i], f[8 * i + 1]), pack2<F16>(f[8 * i + 2], f[8 * i + 3]), pack2<F16>(f[8 * i + 4], f[8 * i + 5]),
                          pack2<F16>(f[8 * i + 6], f[8 * i + 7]));
}
__device__ __forceinline__ void put16(__nv_bfloat16* o, const float* f) { put16_2<false>(o, f); }
__device__ __forceinline__ void put16(__half* o, const float* f) { put16_2<true>(o, f); }

template <typename QT, int MODE>
__global__ void __launch_bounds__(kReadThreads, kReadCtas) rpa_read_kernel(const ReadParams p) {
    __shared__ long long s_page[kReadTokens];  // page and place of a token's slot (page << 32 | place), or -1
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_row = p.D / 16, rows = (p.latent ? 1 : 2) * p.Hkv;
    pdl_trigger();
    pdl_wait();
    const int t_end = (int)((long long)p.T * (blockIdx.x + 1) / gridDim.x);
    for (int t0 = (int)((long long)p.T * blockIdx.x / gridDim.x); t0 < t_end; t0 += kReadTokens) {
        const int n = min(kReadTokens, t_end - t0);
        for (int i = warp; i < n; i += kReadThreads / 32) {
            const int t = t0 + i, s = find_seq(p.cu, p.S, t, lane);
            if (lane != 0) continue;
            long long at = -1;
            if (s >= 0) {
                const int q0 = p.cu[s], ql = p.cu[s + 1] - q0, kl = p.kv_lens[s];
                if (q0 >= 0 && kl <= p.P * p.ps && ql <= kl && q0 + ql <= p.T) {
                    const int j = kl - ql + (t - q0), pg = p.page_indices[(size_t)s * p.P + j / p.ps];
                    if ((unsigned)pg < (unsigned)p.N) at = ((long long)pg << 32) | (j % p.ps);
                    else set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
                }
            }
            s_page[i] = at;
        }
        __syncthreads();
        const int units = n * rows * per_row;
        for (int u0 = tid; u0 < units; u0 += kReadFly * kReadThreads) {
            Unit16<MODE> x[kReadFly];
#pragma unroll
            for (int b = 0; b < kReadFly; ++b) {
                const int u = u0 + b * kReadThreads;
                const int place = u % per_row, i = u / per_row % n, r = u / per_row / n;  // (rows past the last: not loaded)
                const long long slot = u < units ? s_page[i] : -1;
                if (slot < 0) continue;
                const int page = (int)(slot >> 32), at = (int)slot, h = r < p.Hkv ? r : r - p.Hkv, is_v = r >= p.Hkv;
                if constexpr (MODE == kRead4) {
                    const uint8_t* block = p.kv + ((size_t)page * p.Hkv + h) * ((size_t)p.ps * int4_key_bytes(p.D, p.group));
                    const size_t line = (size_t)(is_v ? p.ps : 0) + at;
                    x[b].codes = *reinterpret_cast<const uint2*>(block + line * (p.D / 2) + int4_chunk(place / 2, at, p.D) * 16 +
                                                                 (place & 1) * 8);
                    x[b].scale_zero = reinterpret_cast<const uint32_t*>(block + (size_t)p.ps * p.D)[line * (p.D / p.group) +
                                                                                                    16 * place / p.group];
                } else {
                    const size_t row = ((size_t)page * p.ps + at) * rows + (p.latent ? h : 2 * h + is_v);
                    const uint4* s = reinterpret_cast<const uint4*>(p.kv + (row * p.D + 16 * place) * (MODE == kRead16 ? 2 : 1));
#pragma unroll
                    for (int k = 0; k < (MODE == kRead16 ? 2 : 1); ++k) x[b].a[k] = s[k];
                }
            }
#pragma unroll
            for (int b = 0; b < kReadFly; ++b) {
                const int u = u0 + b * kReadThreads;
                const int place = u % per_row, i = u / per_row % n, r = u / per_row / n;
                if (u >= units || s_page[i] < 0) continue;
                const int h = r < p.Hkv ? r : r - p.Hkv, is_v = r >= p.Hkv;
                float f[16];
                if constexpr (MODE == kRead4) {
                    const float2 sz = f16x2_to_f32x2(x[b].scale_zero);
                    const uint32_t w[2] = {x[b].codes.x, x[b].codes.y};
#pragma unroll
                    for (int k = 0; k < 16; ++k)  // 2^23 + code, exactly
                        f[k] = fmaf(__uint_as_float(((w[k / 8] >> (4 * (k % 8))) & 15u) | 0x4b000000u) - 8388608.f, sz.x, sz.y);
                } else if constexpr (MODE == kRead16) {
                    const uint32_t w[8] = {x[b].a[0].x, x[b].a[0].y, x[b].a[0].z, x[b].a[0].w, x[b].a[1].x, x[b].a[1].y, x[b].a[1].z, x[b].a[1].w};
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 v = p.kt == KT_F16 ? f16x2_to_f32x2(w[k])
                                                        : make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
                        f[2 * k] = v.x;
                        f[2 * k + 1] = v.y;
                    }
                } else {
                    const uint32_t w[4] = {x[b].a[0].x, x[b].a[0].y, x[b].a[0].z, x[b].a[0].w};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint4 v = p.kt == KT_I8     ? cvt8x8_to_f16x8<KT_I8>(w[2 * k], w[2 * k + 1])
                                        : p.kt == KT_E5M2 ? cvt8x8_to_f16x8<KT_E5M2>(w[2 * k], w[2 * k + 1])
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
                const float sc = is_v ? p.v_scale : p.k_scale;
                if (sc != 1.f) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) f[k] *= sc;
                }
                put16(reinterpret_cast<QT*>(is_v ? p.v : p.k) + ((size_t)(t0 + i) * p.Hkv + h) * p.D + 16 * place, f);
            }
        }
        __syncthreads();  // the slots are looked up anew
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
    // a token a CTA at least; without tokens one CTA still checks the lengths
    const int most = sms * kReadCtas, grid = p.T < 1 ? 1 : p.T < most ? p.T : most;
    return q_dtype == RPA_DT_F32   ? launch_as<float>(p, grid, st)
           : q_dtype == RPA_DT_F16 ? launch_as<__half>(p, grid, st)
                                   : launch_as<__nv_bfloat16>(p, grid, st);
}

}  // namespace rpa
