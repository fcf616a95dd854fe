// rpa_weigh.cu -- the softmax weight every cached key receives.
//
//   scores[j] += sum over rows r (query tokens x heads of the group) of 2^(x_rj - M_r) / L_r
//
// x_rj = log2(e) * logit, M_r and L_r the row's maximum and sum over all keys it sees.  A key's weight
// needs L_r, which needs every key: two passes over the logits.  Three launches:
//
//   plan     one CTA: checks the lengths, cuts every sequence into pieces of keys
//   stats    item = (sequence, kv head, block of 16 rows, piece): x = q K^T on warp MMAs; the piece's
//            maxima and sums; the block's last piece to finish merges them, in piece order.  Where a
//            sequence has one block of rows (decode), x itself goes to the workspace.
//   weigh    item = (sequence, kv head, piece): reads x back, or with more blocks computes it again
//            (K from L2), and adds the weights' sum to the scores
//
// Decode is bound by reading K: 2 D bytes a key and head, beside which x is 4 G bytes (6 % at D 128,
// G 4) and stays in L2, where a second pass over K would double the traffic.  S^T = K Q^T: 16 keys on
// the MMA's M side, 8 rows on N.  K goes from global memory straight into the operand registers: the
// contraction may take its terms in any order, so a thread's 16-byte load (8 or 16 neighbouring
// elements of one key) is dealt to its own places of consecutive MMAs, and Q is dealt the same way.
// No shared memory, no barrier in the key loop, the next tile's loads in flight behind this one's MMAs.
//
// Maxima, sums and weights are 32-bit; the products are exact (16-bit operands, 32-bit accumulator)
// where q has the operands' type; q of another type is rounded to it as rpa_forward does.
#include "rpa_evict.cuh"

namespace rpa {

namespace {

constexpr int kWarps = kWeighThreads / 32;

// The first key, rounded down to a piece boundary, that a sequence's first query token sees: pieces start there.
__device__ __forceinline__ int first_key(const WeighParams& p, int kl, int ql) {
    return p.has_window ? max(0, kl - ql - p.window + 1) & ~(kWeighAlign - 1) : 0;
}

// ---------------------------------------------------------------- plan
__global__ void __launch_bounds__(512) rpa_weigh_plan_kernel(const WeighParams p) {
    __shared__ unsigned long long s_sum[512];
    __shared__ long long s_part[512][4];
    __shared__ int s_bad;
    const int tid = threadIdx.x, n = blockDim.x;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) s_bad = 0;
    __syncthreads();
    // a thread's sequences are neighbours
    const int per = (p.S + n - 1) / n, s_lo = min(p.S, tid * per), s_hi = min(p.S, s_lo + per);
    unsigned long long keys = 0;
    for (int s = s_lo; s < s_hi; ++s) {
        const int q0 = p.cu[s], q1 = p.cu[s + 1], kl = p.kv_lens[s];
        if (q0 < 0 || q1 < q0 || kl < 0 || kl > p.P * p.ps || q1 - q0 > kl || q1 > p.T) {
            s_bad = 1;
            break;
        }
        const long long blocks = ((long long)(q1 - q0) * p.G + kWeighRows - 1) / kWeighRows;
        keys += (unsigned long long)(blocks * (kl - first_key(p, kl, q1 - q0))) * p.Hkv;
    }
    s_sum[tid] = keys;
    __syncthreads();
    if (s_bad) {
        if (tid == 0) {
            p.ctrl[0] = p.ctrl[1] = p.ctrl[2] = 0;
            set_status(p.status, RPA_ERR_BAD_LENGTHS);
        }
        return;
    }
    for (int o = n / 2; o > 0; o >>= 1) {
        if (tid < o) s_sum[tid] += s_sum[tid + o];
        __syncthreads();
    }
    const unsigned long long want = s_sum[0] / (unsigned long long)p.target;
    const int chunk = (int)min((want / kWeighAlign + 1) * kWeighAlign, 1ull << 30);
    // per sequence: pieces, then stat items, weight items, row blocks and logits
    auto of = [&](int s, long long (&v)[4]) {
        const int ql = p.cu[s + 1] - p.cu[s], kl = p.kv_lens[s], n_keys = kl - first_key(p, kl, ql);
        const long long rows = (long long)ql * p.G, blocks = (rows + kWeighRows - 1) / kWeighRows * p.Hkv;
        long long pieces = ((long long)n_keys + chunk - 1) / chunk;
        pieces = min(pieces, (long long)p.max_pieces);
        if (rows == 0) pieces = 0;
        v[0] = blocks * pieces;
        v[1] = pieces * p.Hkv;
        v[2] = blocks;
        v[3] = rows <= kWeighRows ? (long long)n_keys * p.Hkv * ((rows + 1) & ~1ll) : 0;
    };
    long long mine[4] = {0, 0, 0, 0};
    for (int s = s_lo; s < s_hi; ++s) {
        long long v[4];
        of(s, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) mine[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s_part[tid][i] = mine[i];
    __syncthreads();
    for (int o = 1; o < n; o <<= 1) {
        long long v[4] = {0, 0, 0, 0};
        if (tid >= o) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = s_part[tid - o][i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) s_part[tid][i] += v[i];
        __syncthreads();
    }
    long long at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = s_part[tid][i] - mine[i];
    for (int s = s_lo; s < s_hi; ++s) {
        long long v[4];
        of(s, v);
        p.stat0[s] = (int)at[0];
        p.item0[s] = (int)at[1];
        p.block0[s] = (int)at[2];
        p.logit0[s] = v[3] > 0 && at[3] + v[3] <= p.max_logits ? at[3] : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) at[i] += v[i];
    }
    const int blocks = (int)s_part[n - 1][2];
    for (int i = tid; i < blocks; i += n) p.done[i] = 0;
    if (tid == 0) {
        p.stat0[p.S] = p.ctrl[0] = (int)s_part[n - 1][0];
        p.item0[p.S] = p.ctrl[1] = (int)s_part[n - 1][1];
        p.block0[p.S] = blocks;
        p.ctrl[2] = chunk;
    }
}

// ---------------------------------------------------------------- logits
// Dealing of a row's elements to the threads of a quad (lane % 4): thread c holds, of every 4 E
// elements, the E from c E on -- one 16-byte load of K (E = 8 two-byte or 16 one-byte elements).
template <int D, int KT>
struct Deal {
    static constexpr int E = kt_8bit(KT) ? 16 : 8;
    static constexpr int LOADS = D / (4 * E);   // 16-byte loads of one key by one thread
    static constexpr int REGS = D / 8;          // 32-bit operand registers of one row's share
};

// One thread's share of query row `row` (tokens x heads of group h) of a sequence, in the operand type.
template <int D, int KT>
__device__ __forceinline__ void load_q(const WeighParams& p, int q0, int h, int row, int rows, int c, uint32_t* r) {
    using L = Deal<D, KT>;
    if (row >= rows) {
#pragma unroll
        for (int i = 0; i < L::REGS; ++i) r[i] = 0;
        return;
    }
    const int i = p.group.div(row), g = row - i * p.G;
    const uint8_t* src = p.q + (((size_t)(q0 + i) * p.Hq + (size_t)h * p.G + g) * D + c * L::E) * 2;
#pragma unroll
    for (int b = 0; b < L::LOADS; ++b)
#pragma unroll
        for (int k = 0; k < L::E / 8; ++k) {
            uint4 v = *reinterpret_cast<const uint4*>(src + (size_t)(b * 4 * L::E + 8 * k) * 2);
            if (kt_8bit(KT) && p.q_bf16) {
                v.x = bf16x2_to_f16x2(v.x);
                v.y = bf16x2_to_f16x2(v.y);
                v.z = bf16x2_to_f16x2(v.z);
                v.w = bf16x2_to_f16x2(v.w);
            }
            uint32_t* d = r + b * (L::E / 2) + 4 * k;
            d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
        }
}

// A 16-key tile: this thread's shares of keys `lane / 4` and `lane / 4 + 8`, as stored.
template <int D, int KT>
struct KeyTile {
    uint4 v[2][Deal<D, KT>::LOADS];
    bool ok[2];   // the key is one of [0, kv_end) on a page that exists
};
template <int D, int KT>
__device__ __forceinline__ void load_k(const WeighParams& p, const int* table, int h, int k0, int k_end, int lane, KeyTile<D, KT>& t) {
    using L = Deal<D, KT>;
    constexpr int EB = kt_8bit(KT) ? 1 : 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int j = k0 + lane / 4 + 8 * i;
        t.ok[i] = j < k_end;
        int pg = 0, at = 0;
        if (t.ok[i]) {
            const int lp = p.page.div(j);
            pg = __ldg(table + lp);
            at = j - lp * p.ps;
            if ((unsigned)pg >= (unsigned)p.N) {
                set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
                t.ok[i] = false;
            }
        }
        const uint8_t* src = p.kv + (((size_t)pg * p.ps + at) * 2 * p.Hkv + 2 * h) * (size_t)(D * EB) + (lane % 4) * 16;
#pragma unroll
        for (int b = 0; b < L::LOADS; ++b) t.v[i][b] = t.ok[i] ? *reinterpret_cast<const uint4*>(src + b * 64) : make_uint4(0, 0, 0, 0);
    }
}

// acc += the tile's 16 keys x 8 rows: acc[0], [1] key lane / 4, rows 2 (lane % 4) and + 1; [2], [3] key + 8
template <int D, int KT>
__device__ __forceinline__ void tile_dot(const KeyTile<D, KT>& t, const uint32_t* q, float* acc) {
    using L = Deal<D, KT>;
    constexpr bool F16 = kt_f16_mma(KT);
#pragma unroll
    for (int b = 0; b < L::LOADS; ++b) {
        if constexpr (kt_8bit(KT)) {
            const uint4 lo0 = cvt8x8_to_f16x8<KT>(t.v[0][b].x, t.v[0][b].y), lo1 = cvt8x8_to_f16x8<KT>(t.v[0][b].z, t.v[0][b].w);
            const uint4 hi0 = cvt8x8_to_f16x8<KT>(t.v[1][b].x, t.v[1][b].y), hi1 = cvt8x8_to_f16x8<KT>(t.v[1][b].z, t.v[1][b].w);
            const uint32_t a0[4] = {lo0.x, hi0.x, lo0.y, hi0.y}, a1[4] = {lo0.z, hi0.z, lo0.w, hi0.w};
            const uint32_t a2[4] = {lo1.x, hi1.x, lo1.y, hi1.y}, a3[4] = {lo1.z, hi1.z, lo1.w, hi1.w};
            mma16816<F16>(acc, a0, q[8 * b], q[8 * b + 1]);
            mma16816<F16>(acc, a1, q[8 * b + 2], q[8 * b + 3]);
            mma16816<F16>(acc, a2, q[8 * b + 4], q[8 * b + 5]);
            mma16816<F16>(acc, a3, q[8 * b + 6], q[8 * b + 7]);
        } else {
            const uint4 lo = t.v[0][b], hi = t.v[1][b];
            const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
            mma16816<F16>(acc, a0, q[4 * b], q[4 * b + 1]);
            mma16816<F16>(acc, a1, q[4 * b + 2], q[4 * b + 3]);
        }
    }
}

// x in the log2 domain; keys the row does not see are -infinity
__device__ __forceinline__ float logit(const WeighParams& p, float dot, int j, int pos, bool ok) {
    const float x = p.has_cap ? p.cap_log2 * tanhf(dot * p.cap_arg) : dot * p.qk_log2;
    const bool sees = ok && (!p.causal || j <= pos) && (!p.has_window || j > pos - p.window);
    return sees ? x : -INFINITY;
}

// A sequence's keys that the rows at positions [p_lo, p_hi] see: [lo, hi)
__device__ __forceinline__ void seen_keys(const WeighParams& p, int kl, int p_lo, int p_hi, int& lo, int& hi) {
    hi = p.causal ? min(kl, p_hi + 1) : kl;
    lo = p.has_window ? max(0, p_lo - p.window + 1) : 0;
}

struct Piece {
    int s, h, piece, pieces, base, k_lo, k_hi, q0, ql, kl;
};
// Piece `piece` of a sequence's keys from `base` on (pieces are equal multiples of kWeighAlign keys, the last the rest)
__device__ __forceinline__ void cut(const WeighParams& p, Piece& c) {
    c.base = first_key(p, c.kl, c.ql);
    const long long len = ((c.kl - c.base + c.pieces - 1) / c.pieces + kWeighAlign - 1) / kWeighAlign * kWeighAlign;
    c.k_lo = (int)min((long long)c.kl, c.base + c.piece * len);
    c.k_hi = (int)min((long long)c.kl, c.k_lo + len);
}

// ---------------------------------------------------------------- stats
// NB: n8 blocks of rows a pass takes (1: at most 8 rows)
template <int D, int KT, int NB>
__device__ __forceinline__ void stat_item(const WeighParams& p, const Piece& c, int rb, float2* s_ml) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, quad = lane % 4;
    const int rows = c.ql * p.G, row0 = rb * kWeighRows;
    const int pos0 = c.kl - c.ql;
    const int n_rows = min(kWeighRows, rows - row0);
    const long long lo0 = p.logit0[c.s];
    const int rs = (rows + 1) & ~1;  // floats of a key's logits
    float* x_out = lo0 >= 0 ? p.logits + lo0 + (size_t)c.h * (c.kl - c.base) * rs : nullptr;
    uint32_t q[NB][Deal<D, KT>::REGS];
#pragma unroll
    for (int b = 0; b < NB; ++b) load_q<D, KT>(p, c.q0, c.h, row0 + 8 * b + lane / 4, rows, quad, q[b]);
    int pos[NB][2];
    float m[NB][2], l[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            pos[b][i] = pos0 + p.group.div(min(row0 + 8 * b + 2 * quad + i, rows - 1));
            m[b][i] = -INFINITY;
            l[b][i] = 0.f;
        }
    int lo, hi;
    seen_keys(p, c.kl, pos0 + p.group.div(row0), pos0 + p.group.div(row0 + n_rows - 1), lo, hi);
    // tiles of the piece that some row sees (all of them where there is one block of rows)
    const int k_first = max(c.k_lo, lo & ~(kWeighAlign - 1)), k_last = min(c.k_hi, hi);
    const int* table = p.page_indices + (size_t)c.s * p.P;
    auto use = [&](const KeyTile<D, KT>& t, int k0) {
        float acc[NB][4];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0.f;
            tile_dot<D, KT>(t, q[b], acc[b]);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[b][e] = logit(p, acc[b][e], k0 + lane / 4 + 8 * (e >> 1), pos[b][e & 1], t.ok[e >> 1]);
            if (x_out) {
                const int r = 8 * b + 2 * quad;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = k0 + lane / 4 + 8 * i;
                    if (j < k_last && r < rs)
                        *reinterpret_cast<float2*>(x_out + (size_t)(j - c.base) * rs + r) = make_float2(acc[b][2 * i], acc[b][2 * i + 1]);
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x0 = acc[b][i], x1 = acc[b][2 + i];
                const float mn = fmaxf(m[b][i], fmaxf(x0, x1));
                if (mn != -INFINITY) {
                    l[b][i] = l[b][i] * ex2(m[b][i] - mn) + (ex2(x0 - mn) + ex2(x1 - mn));
                    m[b][i] = mn;
                }
            }
        }
    };
    // a second tile's loads in flight where its registers, and the rows' operands, leave 48 of 128 for the rest
    constexpr bool kAhead = 2 * 8 * Deal<D, KT>::LOADS + NB * Deal<D, KT>::REGS <= 80;
    int k0 = k_first + 16 * warp;
    if constexpr (kAhead) {
        KeyTile<D, KT> a, b;
        if (k0 < k_last) load_k<D, KT>(p, table, c.h, k0, k_last, lane, a);
        while (k0 < k_last) {
            const int k1 = k0 + 16 * kWarps;
            if (k1 < k_last) load_k<D, KT>(p, table, c.h, k1, k_last, lane, b);
            use(a, k0);
            k0 = k1 + 16 * kWarps;
            if (k0 < k_last) load_k<D, KT>(p, table, c.h, k0, k_last, lane, a);
            if (k1 < k_last) use(b, k1);
        }
    } else {
        for (; k0 < k_last; k0 += 16 * kWarps) {
            KeyTile<D, KT> a;
            load_k<D, KT>(p, table, c.h, k0, k_last, lane, a);
            use(a, k0);
        }
    }
    // the piece's maximum and sum of each row: over a warp's keys, then over the warps
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mm = m[b][i], ll = l[b][i];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, mm, o), l2 = __shfl_xor_sync(0xffffffffu, ll, o);
                const float mn = fmaxf(mm, m2);
                if (mn != -INFINITY) ll = ll * ex2(mm - mn) + l2 * ex2(m2 - mn);
                mm = mn;
            }
            if (lane < 4) s_ml[warp * kWeighRows + 8 * b + 2 * lane + i] = make_float2(mm, ll);
        }
    __syncthreads();
    const int nb = (rows + kWeighRows - 1) / kWeighRows;
    const int block = p.block0[c.s] + c.h * nb + rb;
    float2* part = p.part + (size_t)block * p.max_pieces * kWeighRows;
    __shared__ int s_last;
    if (warp == 0) {
        if (lane < n_rows) {
            float mm = -INFINITY, ll = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float2 v = s_ml[w * kWeighRows + lane];
                const float mn = fmaxf(mm, v.x);
                if (mn != -INFINITY) ll = ll * ex2(mm - mn) + v.y * ex2(v.x - mn);
                mm = mn;
            }
            part[c.piece * kWeighRows + lane] = make_float2(mm, ll);
        }
        __threadfence();
        __syncwarp();
        if (lane == 0) s_last = atomicAdd(p.done + block, 1) == c.pieces - 1;
        __syncwarp();
    }
    __syncthreads();
    // the block's last piece merges all of them, each row's in piece order
    if (s_last) {
        __threadfence();
        for (int r = warp; r < n_rows; r += kWarps) {
            float mm = -INFINITY, ll = 0.f;
            for (int k = lane; k < c.pieces; k += 32) {
                const float2 v = __ldcg(part + k * kWeighRows + r);
                const float mn = fmaxf(mm, v.x);
                if (mn != -INFINITY) ll = ll * ex2(mm - mn) + v.y * ex2(v.x - mn);
                mm = mn;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, mm, o), l2 = __shfl_xor_sync(0xffffffffu, ll, o);
                const float mn = fmaxf(mm, m2);
                if (mn != -INFINITY) ll = ll * ex2(mm - mn) + l2 * ex2(m2 - mn);
                mm = mn;
            }
            if (lane == 0) {
                const int row = row0 + r, g = row - p.group.div(row) * p.G;
                ll = add_sink(ll, p.sinks, c.h * p.G + g, mm);
                // a row that sees nothing gives nothing
                p.stat[(size_t)block * kWeighRows + r] = mm == -INFINITY ? make_float2(0.f, 0.f) : make_float2(mm, 1.f / ll);
            }
        }
    }
    __syncthreads();  // s_ml and s_last are free again
}

template <int D, int KT>
__global__ void __launch_bounds__(kWeighThreads, D == 256 ? 1 : 2) rpa_weigh_stats_kernel(const WeighParams p) {
    __shared__ float2 s_ml[kWarps * kWeighRows];
    pdl_trigger();
    pdl_wait();
    const int items = p.ctrl[0], lane = threadIdx.x & 31;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        // items of a sequence: piece, then row block, then kv head (neighbours read neighbouring rows)
        Piece c;
        c.s = find_seq(p.stat0, p.S, it, lane);
        c.q0 = p.cu[c.s];
        c.ql = p.cu[c.s + 1] - c.q0;
        c.kl = p.kv_lens[c.s];
        const int at = it - p.stat0[c.s], nb = (c.ql * p.G + kWeighRows - 1) / kWeighRows;
        c.pieces = (p.stat0[c.s + 1] - p.stat0[c.s]) / (nb * p.Hkv);
        c.h = at % p.Hkv;
        const int rb = at / p.Hkv % nb;
        c.piece = at / p.Hkv / nb;
        cut(p, c);
        if (min(kWeighRows, c.ql * p.G - rb * kWeighRows) <= 8) stat_item<D, KT, 1>(p, c, rb, s_ml);
        else stat_item<D, KT, 2>(p, c, rb, s_ml);
    }
}

// ---------------------------------------------------------------- weigh
__device__ __forceinline__ void add_score(const WeighParams& p, const int* table, int h, int j, int fresh, float w) {
    const int lp = p.page.div(j), pg = __ldg(table + lp);
    if ((unsigned)pg >= (unsigned)p.N) return;
    float* dst = p.scores + ((size_t)pg * p.Hkv + h) * p.ps + (j - lp * p.ps);
    // the call's own keys start from 0; the others add (a page may be shared by sequences)
    if (j >= fresh) *dst = w;
    else atomicAdd(dst, w);
}

template <int D, int KT>
__global__ void __launch_bounds__(kWeighThreads) rpa_weigh_kernel(const WeighParams p) {
    __shared__ float2 s_stat[kWeighRows];
    pdl_trigger();
    pdl_wait();
    const int items = p.ctrl[1], tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int it = blockIdx.x; it < items; it += gridDim.x) {
        Piece c;
        c.s = find_seq(p.item0, p.S, it, lane);
        c.q0 = p.cu[c.s];
        c.ql = p.cu[c.s + 1] - c.q0;
        c.kl = p.kv_lens[c.s];
        c.pieces = (p.item0[c.s + 1] - p.item0[c.s]) / p.Hkv;
        const int at = it - p.item0[c.s];
        c.h = at % p.Hkv;
        c.piece = at / p.Hkv;
        cut(p, c);
        const int rows = c.ql * p.G, nb = (rows + kWeighRows - 1) / kWeighRows, pos0 = c.kl - c.ql;
        const int* table = p.page_indices + (size_t)c.s * p.P;
        const float2* stat = p.stat + (size_t)(p.block0[c.s] + c.h * nb) * kWeighRows;
        int lo, hi;
        seen_keys(p, c.kl, pos0, c.kl - 1, lo, hi);
        const int k_lo = max(c.k_lo, lo);
        const long long lo0 = p.logit0[c.s];
        if (lo0 >= 0) {
            __syncthreads();
            if (tid < kWeighRows) s_stat[tid] = tid < rows ? stat[tid] : make_float2(0.f, 0.f);
            __syncthreads();
            const int rs = (rows + 1) & ~1;
            const float* x = p.logits + lo0 + (size_t)c.h * (c.kl - c.base) * rs;
            for (int j = k_lo + tid; j < c.k_hi; j += kWeighThreads) {
                float w = 0.f;
                for (int r = 0; r < rs; r += 2) {
                    const float2 v = *reinterpret_cast<const float2*>(x + (size_t)(j - c.base) * rs + r);
                    w += ex2(v.x - s_stat[r].x) * s_stat[r].y;
                    if (r + 1 < rows) w += ex2(v.y - s_stat[r + 1].x) * s_stat[r + 1].y;
                }
                add_score(p, table, c.h, j, pos0, w);
            }
        } else {
            const int quad = lane % 4;
            for (int k0 = (k_lo & ~15) + 16 * warp; k0 < c.k_hi; k0 += 16 * kWarps) {
                KeyTile<D, KT> t;
                load_k<D, KT>(p, table, c.h, k0, c.k_hi, lane, t);
                float w0 = 0.f, w1 = 0.f;
                // rows whose tokens see the tile: from the first token at or behind its first key
                int r_lo = 0, r_hi = rows;
                if (p.causal) r_lo = max(0, k0 - pos0) * p.G & ~7;
                if (p.has_window) r_hi = min((long long)rows, max(0ll, (long long)k0 + 15 + p.window - pos0) * p.G);
                for (int r0 = r_lo; r0 < r_hi; r0 += 8) {
                    uint32_t q[Deal<D, KT>::REGS];
                    load_q<D, KT>(p, c.q0, c.h, r0 + lane / 4, rows, quad, q);
                    float acc[4] = {0.f, 0.f, 0.f, 0.f};
                    tile_dot<D, KT>(t, q, acc);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int r = r0 + 2 * quad + i;
                        if (r >= rows) continue;
                        const float2 st = stat[r];
                        const int pos = pos0 + p.group.div(r);
                        w0 += ex2(logit(p, acc[i], k0 + lane / 4, pos, t.ok[0]) - st.x) * st.y;
                        w1 += ex2(logit(p, acc[2 + i], k0 + lane / 4 + 8, pos, t.ok[1]) - st.x) * st.y;
                    }
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    w0 += __shfl_xor_sync(0xffffffffu, w0, o);
                    w1 += __shfl_xor_sync(0xffffffffu, w1, o);
                }
                const int j = k0 + lane / 4 + 8 * quad;
                if (quad < 2 && j >= k_lo && j < c.k_hi) add_score(p, table, c.h, j, pos0, quad ? w1 : w0);
            }
        }
    }
}

template <int D, int KT>
struct WeighKern {
    static cudaError_t prepare(int* bps) {
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(bps, rpa_weigh_stats_kernel<D, KT>, kWeighThreads, 0);
    }
    static cudaError_t launch(const WeighParams& p, int grid, cudaStream_t st) {
        cudaError_t e = launch_pdl(rpa_weigh_plan_kernel, 1, 512, 0, st, p);
        if (e == cudaSuccess) e = launch_pdl(rpa_weigh_stats_kernel<D, KT>, grid, kWeighThreads, 0, st, p);
        if (e == cudaSuccess) e = launch_pdl(rpa_weigh_kernel<D, KT>, grid, kWeighThreads, 0, st, p);
        return e;
    }
};

template <int D, typename Op>
cudaError_t weigh_types(int kt, Op op) {
    switch (kt) {
        case KT_BF16: return op(WeighKern<D, KT_BF16>{});
        case KT_F16: return op(WeighKern<D, KT_F16>{});
        case KT_E4M3: return op(WeighKern<D, KT_E4M3>{});
        case KT_E5M2: return op(WeighKern<D, KT_E5M2>{});
        default: return op(WeighKern<D, KT_I8>{});
    }
}
template <typename Op>
cudaError_t weigh_dispatch(int D, int kt, Op op) {
    return D == 64 ? weigh_types<64>(kt, op) : D == 128 ? weigh_types<128>(kt, op) : weigh_types<256>(kt, op);
}

}  // namespace

cudaError_t weigh_prepare(int D, int kt, int* bps) {
    return weigh_dispatch(D, kt, [&](auto k) { return decltype(k)::prepare(bps); });
}
cudaError_t launch_weigh(const WeighParams& p, int kt, int grid, cudaStream_t st) {
    return weigh_dispatch(p.D, kt, [&](auto k) { return decltype(k)::launch(p, grid, st); });
}

}  // namespace rpa
