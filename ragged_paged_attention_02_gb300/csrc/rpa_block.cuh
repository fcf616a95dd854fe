// rpa_block.cuh -- block-wide scans and reductions of the planners.
#pragma once

#include "rpa_internal.cuh"

namespace rpa {

// Exclusive scan of N ints per thread over the whole block (one pass for all N): r gets the
// thread's offsets, tot the block's sums.  s_scan holds 33 N ints.
template <int N>
__device__ __forceinline__ void block_scan(const int (&v)[N], int (&r)[N], int (&tot)[N], int* s_scan) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int nwarps = blockDim.x >> 5;
    int x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = v[i];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int y = __shfl_up_sync(0xffffffffu, x[i], o);
            if (lane >= o) x[i] += y;
        }
    }
    if (lane == 31) {
#pragma unroll
        for (int i = 0; i < N; ++i) s_scan[warp * N + i] = x[i];
    }
    __syncthreads();
    if (warp == 0) {
        int w[N], ww[N];
#pragma unroll
        for (int i = 0; i < N; ++i) ww[i] = w[i] = lane < nwarps ? s_scan[lane * N + i] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int y = __shfl_up_sync(0xffffffffu, ww[i], o);
                if (lane >= o) ww[i] += y;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            s_scan[lane * N + i] = ww[i] - w[i];
            if (lane == 31) s_scan[32 * N + i] = ww[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        r[i] = x[i] - v[i] + s_scan[warp * N + i];
        tot[i] = s_scan[32 * N + i];
    }
    __syncthreads();
}

// Sums of two 64-bit values per thread over the block (all threads get them).  s_red holds 64.
__device__ __forceinline__ void block_sum64x2(unsigned long long& a, unsigned long long& b, unsigned long long* s_red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if (lane == 0) {
        s_red[warp] = a;
        s_red[32 + warp] = b;
    }
    __syncthreads();
    unsigned long long x = lane < nwarps ? s_red[lane] : 0ull, y = lane < nwarps ? s_red[32 + lane] : 0ull;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    __syncthreads();
    a = x;
    b = y;
}
// Minimum of one 64-bit value per thread over the block (all threads get it).  s_red holds 32.
__device__ __forceinline__ unsigned long long block_min64(unsigned long long v, unsigned long long* s_red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
        v = w < v ? w : v;
    }
    if (lane == 0) s_red[warp] = v;
    __syncthreads();
    unsigned long long t = lane < nwarps ? s_red[lane] : ~0ull;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long w = __shfl_xor_sync(0xffffffffu, t, o);
        t = w < t ? w : t;
    }
    __syncthreads();
    return t;
}

// first s in [0, n) with ends[s] > u (ends non-decreasing, ends[n-1] > u)
__device__ __forceinline__ int upper_seq(const int* ends, int n, int u) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        int mid = (lo + hi) >> 1;
        if (ends[mid] > u) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

}  // namespace rpa
