// rpa_weigh.cu -- the softmax weight every cached key receives.
//
//   scores[j] += sum over rows r (query tokens x heads of the group) of 2^(x_rj - S_r),  S_r = M_r + log2 L_r
//
// x_rj = log2(e) * logit, M_r and L_r the row's maximum and sum over all keys it sees.  A key's weight
// needs L_r, which needs every key: two passes over the logits.  Three launches:
//
//   plan     one CTA: checks the lengths, cuts every sequence into pieces of keys
//   stats    item = (sequence, kv head, block of 16 rows, piece): x = q K^T on warp MMAs, maxima and
//            sums; a block's last warp to finish merges all of them, in order.  Where a sequence has
//            one block of rows (decode), x itself goes to the workspace.
//   weigh    a warp takes (sequence, 1 to 8 kv heads, 128 keys) and reads x back, or with more blocks takes 16 to
//            64 keys and computes it again (K from L2, all row blocks past the keys in its registers),
//            and adds the weights' sum to the scores
//
// Decode is bound by reading K: 2 D bytes a key and head, beside which x is 4 G bytes (6 % at D 128,
// G 4) and stays in L2, where a second pass over K would double the traffic.  S^T = K Q^T: 16 keys on
// the MMA's M side, 8 rows on N.  The contraction may take its terms in any order, so a thread's 16-byte
// load (8 or 16 neighbouring elements of one key) is dealt to its own places of consecutive MMAs, and Q is
// dealt the same way: one load feeds two MMAs, for 16-bit and (through a conversion) for 8-bit K alike.
//
// The stats kernel is persistent, three CTAs an SM: a producer warp looks up items and page ids and copies
// K rows in stages of 64 keys, one bulk tensor copy a page run, into a ring; four warps take 16 keys of a
// stage each and share nothing but the ring.  The copies land in blocks of 64-byte columns, so that the
// eight lanes that a shared-memory access serves at once (four of two neighbouring keys) read 128
// neighbouring bytes.  (Warps that loaded their own keys were bound by their own instructions and waits:
// 16-byte loads into registers read 4.4 TB/s, 16-byte asynchronous copies 4.8, row copies by each lane 3.9.)
//
// 64 decodes over 612 MB of K (32 heads, 8 kv heads, D 128, bf16): 124 us, of which plan 4, stats 109 (5.5 TB/s; its
// copies alone, computing nothing, take 100: K rows are every other 256 bytes) and weigh 11.  The last 202 tokens of six
// prompts of 1 to 6 k keys (16 heads, 8 kv heads, D 64, f16; 1.1 GFLOP): 47.2 us, 4 / 26 / 17: bound by
// instructions, some 300 a warp for a tile of 16 keys x 16 rows, and by a row block's end (1.8 us: reductions, the counter,
// the next item).  Measured there: two or four row blocks a warp over the same keys 50 and 52 us; four CTAs an SM 49.5.
//
// Maxima, sums and weights are 32-bit; the products are exact (16-bit operands, 32-bit accumulator)
// where q has the operands' type; q of another type is rounded to it as rpa_forward does.
#include <type_traits>

#include "rpa_block.cuh"
#include "rpa_evict.cuh"

namespace rpa {

namespace {

constexpr int kWarps = kWeighThreads / 32;
constexpr uint64_t kWeighWaitNs = 1000000000ull;  // bound of a wait for copies; then RPA_ERR_TIMEOUT

// Weigh items of a call: their numbers, and a warp's next one, in 31 bits (sequences may share pages, so that no memory
// bounds their keys)
constexpr unsigned long long kMostItems = (1ull << 31) - (1ull << 20);

// The first key, rounded down to a piece boundary, that a sequence's first query token sees: pieces start there.
__device__ __forceinline__ int first_key(const WeighParams& p, int kl, int ql) {
    return p.has_window ? max(0, kl - ql - p.window + 1) & ~(kWeighAlign - 1) : 0;
}

// ---------------------------------------------------------------- plan
__global__ void __launch_bounds__(kPlanThreads, 1) rpa_weigh_plan_kernel(const WeighParams p) {
    __shared__ int s_scan[33 * 3];
    __shared__ unsigned long long s_red[64];
    __shared__ int s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) s_bad = 0;
    __syncthreads();
    unsigned long long keys = 0, most_items = 0;  // weigh items, if all logits are computed again
    for (int s = tid; s < p.S; s += kPlanThreads) {
        const int q0 = p.cu[s], q1 = p.cu[s + 1], kl = p.kv_lens[s];
        if (q0 < 0 || q1 < q0 || kl < 0 || kl > p.P * p.ps || q1 - q0 > kl || q1 > p.T) {
            s_bad = 1;
        } else {
            const long long blocks = ((long long)(q1 - q0) * p.G + kWeighRows - 1) / kWeighRows;
            const int n_keys = kl - first_key(p, kl, q1 - q0);
            keys += (unsigned long long)(blocks * n_keys) * p.Hkv;
            if (blocks > 0) most_items += (unsigned long long)((n_keys + p.item_keys - 1) / p.item_keys) * p.Hkv;
        }
    }
    block_sum64x2(keys, most_items, s_red);
    if (s_bad || most_items > kMostItems) {
        if (tid == 0) {
            p.ctrl[0] = p.ctrl[1] = p.ctrl[2] = 0;
            set_status(p.status, RPA_ERR_BAD_LENGTHS);
        }
        return;
    }
    // keys of a piece: four pieces a resident CTA, so that uneven ones even out, but not under 512 keys (a piece costs
    // about what 100 keys do) unless that leaves CTAs without any
    const unsigned long long slots = (unsigned long long)p.ctas;
    const unsigned long long want = max(keys / (4 * slots), min(512ull, keys / slots));
    const int chunk = (int)min((want / kWeighAlign + (want % kWeighAlign ? 1 : 0)) * kWeighAlign + (want ? 0 : kWeighAlign), 1ull << 30);
    // kv heads of a weigh item that reads logits back: more where every warp has several items all the same, for what an
    // item looks up takes longer than a head's sums (64 decodes, 7 items a warp: 20, 14.6, 11.8 and 10.7 us with 1, 2, 4, 8)
    const unsigned long long share = keys / kWeighKeys / (unsigned long long)p.weigh_warps;
    const int heads = share >= 4 ? 8 : share >= 2 ? 4 : share >= 1 ? 2 : 1;
    // per sequence: stat items, weigh items, row blocks; and logits
    int n[3] = {0, 0, 0};
    long long n_logits = 0;
    for (int base = 0; base < p.S; base += kPlanThreads) {
        const int s = base + tid;
        int add[3] = {0, 0, 0}, off[3], tot[3], n_keys = 0;
        long long logits = 0, rows = 0;
        if (s < p.S) {
            const int ql = p.cu[s + 1] - p.cu[s], kl = p.kv_lens[s];
            n_keys = kl - first_key(p, kl, ql);
            rows = (long long)ql * p.G;
            // (each sequence's start on 16 bytes)
            if (rows > 0 && rows <= kWeighRows) logits = ((long long)n_keys * p.Hkv * ((rows + 1) & ~1ll) + 3) & ~3ll;
        }
        // where each sequence's logits start: a scan of 64-bit counts
        long long sum = logits;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) s_red[warp] = (unsigned long long)sum;
        __syncthreads();
        long long before = 0, all = 0;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            const long long y = (long long)s_red[w];
            if (w < warp) before += y;
            all += y;
        }
        const long long at = n_logits + before + sum - logits;
        const bool keep = logits > 0 && at + logits <= p.max_logits;
        if (rows > 0) {
            const int pieces = min((n_keys + chunk - 1) / chunk, p.max_pieces), item = keep ? kWeighKeys : p.item_keys;
            add[2] = (int)((rows + kWeighRows - 1) / kWeighRows) * p.Hkv;
            add[0] = add[2] * pieces;
            add[1] = (n_keys + item - 1) / item * (keep ? (p.Hkv + heads - 1) / heads : p.Hkv);
        }
        block_scan<3>(add, off, tot, s_scan);
        if (s < p.S) {
            p.stat0[s] = n[0] + off[0];
            p.item0[s] = n[1] + off[1];
            p.block0[s] = n[2] + off[2];
            p.logit0[s] = keep ? at : -1;
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) n[i] += tot[i];
        n_logits += all;
    }
    for (int i = tid; i < n[2]; i += kPlanThreads) p.done[i] = 0;
    if (tid == 0) {
        p.ctrl[2] = 0;
        p.ctrl[3] = heads;
        p.stat0[p.S] = p.ctrl[0] = n[0];
        p.item0[p.S] = p.ctrl[1] = n[1];
        p.block0[p.S] = n[2];
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

// One thread's share of query row `row` (tokens x heads of group h) of a sequence, in the operand type; behind the last
// row that row again, which brings no infinities or NaN of its own.
template <int D, int KT>
__device__ __forceinline__ void load_q(const WeighParams& p, int q0, int h, int row, int rows, int c, uint32_t* r) {
    using L = Deal<D, KT>;
    row = min(row, rows - 1);
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

// (Not a read-only load: the kernel that writes these rows, an append in front of this call, may still run when this one
// starts.)
__device__ __forceinline__ uint4 load_stream(const uint8_t* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.b32 {%0,%1,%2,%3}, [%4], %5;\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy)
                 : "memory");
    return v;
}
__device__ __forceinline__ uint64_t l2_policy_normal() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;\n" : "=l"(pol));
    return pol;
}

// A 16-key tile: this thread's shares of keys `lane / 4` and `lane / 4 + 8`, as stored.
template <int D, int KT>
struct KeyTile {
    uint4 v[2][Deal<D, KT>::LOADS];
    bool ok[2];   // the key is one of [0, kv_end) on a page that exists
};
template <int D, int KT>
__device__ __forceinline__ void load_k(const WeighParams& p, const int* table, int h, int k0, int k_end, int lane, uint64_t policy,
                                       KeyTile<D, KT>& t) {
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
        for (int b = 0; b < L::LOADS; ++b) t.v[i][b] = t.ok[i] ? load_stream(src + b * 64, policy) : make_uint4(0, 0, 0, 0);
    }
}

// acc += 16 keys x 8 rows over the elements of load b: lo and hi are the thread's shares of keys lane / 4 and + 8.
// acc[0], [1]: key lane / 4, rows 2 (lane % 4) and + 1; [2], [3]: key + 8
template <int KT, int NB, int REGS>
__device__ __forceinline__ void load_dot(const uint4& lo, const uint4& hi, int b, const uint32_t (&q)[NB][REGS], float (&acc)[NB][4]) {
    constexpr bool F16 = kt_f16_mma(KT);
    if constexpr (kt_8bit(KT)) {
        const uint4 lo0 = cvt8x8_to_f16x8<KT>(lo.x, lo.y), lo1 = cvt8x8_to_f16x8<KT>(lo.z, lo.w);
        const uint4 hi0 = cvt8x8_to_f16x8<KT>(hi.x, hi.y), hi1 = cvt8x8_to_f16x8<KT>(hi.z, hi.w);
        const uint32_t a[4][4] = {{lo0.x, hi0.x, lo0.y, hi0.y}, {lo0.z, hi0.z, lo0.w, hi0.w},
                                  {lo1.x, hi1.x, lo1.y, hi1.y}, {lo1.z, hi1.z, lo1.w, hi1.w}};
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) mma16816<F16>(acc[n], a[i], q[n][8 * b + 2 * i], q[n][8 * b + 2 * i + 1]);
    } else {
        const uint32_t a[2][4] = {{lo.x, hi.x, lo.y, hi.y}, {lo.z, hi.z, lo.w, hi.w}};
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) mma16816<F16>(acc[n], a[i], q[n][4 * b + 2 * i], q[n][4 * b + 2 * i + 1]);
    }
}
template <int D, int KT, int NB>
__device__ __forceinline__ void tile_dot(const KeyTile<D, KT>& t, const uint32_t (&q)[NB][Deal<D, KT>::REGS], float (&acc)[NB][4]) {
#pragma unroll
    for (int b = 0; b < Deal<D, KT>::LOADS; ++b) load_dot<KT>(t.v[0][b], t.v[1][b], b, q, acc);
}

// ---- the stats kernel's ring
template <int D, int KT>
struct Ring {
    static constexpr int ROW = D * (kt_8bit(KT) ? 1 : 2);
    static constexpr int KEYS = 64;             // of a stage: 16 a consumer warp
    static constexpr int STAGE = KEYS * ROW;
    // resident an SM: at D 256 two, of 168 registers a thread, else three of 128
    static constexpr int CTAS = D == 256 ? 2 : 3;
    static constexpr int STAGES = ROW == 512 ? 3 : ROW == 256 ? 4 : 6;
    static constexpr int SMEM = STAGES * STAGE + 128;
    static_assert(CTAS * SMEM <= 220 * 1024, "shared memory of an SM");
};
constexpr int kConsumers = 4;
constexpr int kStatThreads = 32 * (kConsumers + 1);

struct Piece {
    int s, h, rb, nb, piece, pieces, base, k_lo, k_hi, q0, ql, kl;
};
// What a stage holds: keys [k0, k0 + 64) of an item, those below k_last; a bit for each page run that is there
struct StageMeta {
    Piece c;
    int k0, k_first, k_last;
    uint32_t runs;
    int stop;
};

__device__ __forceinline__ uint4 read16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

// Soft cap of N products, in the log2 domain.  A function of its own: the inlined tanh would cost the key
// loops their registers.
__device__ __noinline__ float capped(float dot, float arg, float cap_log2) { return cap_log2 * tanhf(dot * arg); }
template <int N>
__device__ __forceinline__ void scale(const WeighParams& p, float (&x)[N]) {
    if (p.has_cap) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = capped(x[i], p.cap_arg, p.cap_log2);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] *= p.qk_log2;
    }
}
// With MASK, keys the row does not see are -infinity
template <bool MASK>
__device__ __forceinline__ float hide(const WeighParams& p, float x, int j, int pos, bool ok) {
    if constexpr (!MASK) return x;
    const bool sees = ok && (!p.causal || j <= pos) && (!p.has_window || j > pos - p.window);
    return sees ? x : -INFINITY;
}
// Whether some of the keys [k0, k1) is hidden from some row at positions [p_lo, p_hi]
__device__ __forceinline__ bool some_hidden(const WeighParams& p, int k0, int k1, int p_lo, int p_hi) {
    return (p.causal && k1 - 1 > p_lo) || (p.has_window && k0 <= p_hi - p.window);
}

// (m, l) of a set of keys joined with another's
__device__ __forceinline__ void join(float& m, float& l, float m2, float l2) {
    const float mn = fmaxf(m, m2);
    if (mn != -INFINITY) l = l * ex2(m - mn) + l2 * ex2(m2 - mn);
    m = mn;
}

// ---------------------------------------------------------------- stats
// Piece `piece` of a sequence's keys from `base` on (pieces are equal multiples of kWeighAlign keys, the last the rest)
__device__ __forceinline__ void cut(const WeighParams& p, Piece& c) {
    c.base = first_key(p, c.kl, c.ql);
    const long long len = ((c.kl - c.base + c.pieces - 1) / c.pieces + kWeighAlign - 1) / kWeighAlign * kWeighAlign;
    c.k_lo = (int)min((long long)c.kl, c.base + c.piece * len);
    c.k_hi = (int)min((long long)c.kl, c.k_lo + len);
}

// Rows of an item's block, positions and the keys some of them sees: [k_first, k_last) of the piece
__device__ __forceinline__ void seen(const WeighParams& p, const Piece& c, int& k_first, int& k_last) {
    const int row0 = c.rb * kWeighRows, n_rows = min(kWeighRows, c.ql * p.G - row0), pos0 = c.kl - c.ql;
    const int p_lo = pos0 + p.group.div(row0), p_hi = pos0 + p.group.div(row0 + n_rows - 1);
    const int hi = p.causal ? min(c.kl, p_hi + 1) : c.kl, lo = p.has_window ? max(0, p_lo - p.window + 1) : 0;
    k_first = max(c.k_lo, lo & ~(kWeighAlign - 1));
    k_last = min(c.k_hi, hi);
}

// A consumer warp's work on one item, from its first stage (already full) to its last.  NB: n8 blocks of rows.
template <int D, int KT, int NB>
__device__ __forceinline__ bool stat_item(const WeighParams& p, const StageMeta* meta, uint32_t ring, uint32_t full, uint32_t empty,
                                          int warp, int& st, uint32_t& phase) {
    using R = Ring<D, KT>;
    constexpr int LOADS = Deal<D, KT>::LOADS;
    using Acc = float[NB][4];
    const int lane = threadIdx.x & 31, quad = lane % 4;
    const Piece& c = meta[st].c;  // until the stage is freed
    const int k_first = meta[st].k_first, k_last = meta[st].k_last, base = c.base;
    const int rows = c.ql * p.G, row0 = c.rb * kWeighRows, pos0 = c.kl - c.ql, head0 = c.h * p.G;
    const int n_rows = min(kWeighRows, rows - row0);
    const long long lo0 = p.logit0[c.s];
    const int rs = (rows + 1) & ~1;  // floats of a key's logits
    float* x_out = lo0 >= 0 ? p.logits + lo0 + (size_t)c.h * (c.kl - base) * rs : nullptr;
    const int block = p.block0[c.s] + c.h * c.nb + c.rb, parts = c.pieces * kConsumers, my_part = c.piece * kConsumers + warp;
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
    const int p_lo = pos0 + p.group.div(row0), p_hi = pos0 + p.group.div(row0 + n_rows - 1);
    // where this thread's two keys of a stage sit: run, place in the run; a run is [ROW / 64][BR][64 bytes]
    uint32_t key_at[2], key_run[2];
    const uint32_t column = (uint32_t)p.BR * 64u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int kk = 16 * warp + lane / 4 + 8 * i;
        key_run[i] = (uint32_t)kk >> p.br_shift;
        key_at[i] = key_run[i] * (uint32_t)(p.BR * R::ROW) + (uint32_t)(kk & (p.BR - 1)) * 64u + quad * 16;
    }
    auto finish = [&](auto masked, Acc& acc, uint32_t runs, int kw) {
        constexpr bool MASK = decltype(masked)::value;
        if constexpr (MASK) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = kw + lane / 4 + 8 * (e >> 1);
                    acc[b][e] = hide<true>(p, acc[b][e], j, pos[b][e & 1], j < k_last && (runs >> key_run[e >> 1] & 1u));
                }
        }
        if (x_out) {
            float* x = x_out + (size_t)(kw - base + lane / 4) * rs + 2 * quad;
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int b = 0; b < NB; ++b)
                    if ((!MASK || kw + lane / 4 + 8 * i < k_last) && 8 * b + 2 * quad < rs)
                        *reinterpret_cast<float2*>(x + 8 * i * rs + 8 * b) = make_float2(acc[b][2 * i], acc[b][2 * i + 1]);
        }
        // new maxima; mostly there are none
        bool grow = false;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) grow = grow || fmaxf(acc[b][i], acc[b][2 + i]) > m[b][i];
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mn = fmaxf(m[b][i], fmaxf(acc[b][i], acc[b][2 + i]));
                    if (mn != -INFINITY) l[b][i] *= ex2(m[b][i] - mn);
                    m[b][i] = mn;
                }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // before the first key that is seen there is no maximum: nothing to add
                const float at = m[b][i] == -INFINITY ? 0.f : m[b][i];
                l[b][i] += ex2(acc[b][i] - at) + ex2(acc[b][2 + i] - at);
            }
    };
    for (int k0 = k_first;;) {
        const int kw = k0 + 16 * warp;
        const uint32_t runs = meta[st].runs;
        const uint32_t from = ring + st * R::STAGE;
        const bool any = kw < k_last;
        // the rows go to registers first, and the stage's place back to the producer, where they fit
        constexpr bool kEarly = 8 * LOADS + NB * Deal<D, KT>::REGS <= 48;
        uint4 lo[LOADS], hi[LOADS];
        auto free_stage = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + st * 8);
            if (++st == R::STAGES) {
                st = 0;
                phase ^= 1u;
            }
        };
        if (kEarly) {
            if (any) {
#pragma unroll
                for (int b = 0; b < LOADS; ++b) {
                    lo[b] = read16(from + key_at[0] + b * column);
                    hi[b] = read16(from + key_at[1] + b * column);
                }
            }
            free_stage();
        }
        Acc acc;
        if (any) {
            // two chains of MMAs where there is one block of rows
            float odd[1][4] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
            for (int b = 0; b < LOADS; ++b) {
                if (!kEarly) {
                    lo[b] = read16(from + key_at[0] + b * column);
                    hi[b] = read16(from + key_at[1] + b * column);
                }
                if constexpr (NB == 1) {
                    if (b & 1) load_dot<KT>(lo[b], hi[b], b, q, odd);
                    else load_dot<KT>(lo[b], hi[b], b, q, acc);
                } else {
                    load_dot<KT>(lo[b], hi[b], b, q, acc);
                }
            }
            if (NB == 1) {
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[0][e] += odd[0][e];
            }
#pragma unroll
            for (int n = 0; n < NB; ++n) scale(p, acc[n]);
        }
        if (!kEarly) free_stage();
        if (any) {
            if (runs == p.all_runs && kw + 16 <= k_last && !some_hidden(p, kw, kw + 16, p_lo, p_hi)) finish(std::false_type{}, acc, runs, kw);
            else finish(std::true_type{}, acc, runs, kw);
        }
        k0 += R::KEYS;
        if (k0 >= k_last) break;
        if (!mbar_wait(full + st * 8, phase, p.status, kWeighWaitNs)) return false;
    }
    // the warp's maximum and sum of each row, over the lanes that hold its keys
    float2* part = p.part + (size_t)block * (p.max_pieces * kConsumers) * kWeighRows;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, m[b][i], o), l2 = __shfl_xor_sync(0xffffffffu, l[b][i], o);
                join(m[b][i], l[b][i], m2, l2);
            }
            if (lane < 4) part[my_part * kWeighRows + 8 * b + 2 * lane + i] = make_float2(m[b][i], l[b][i]);
        }
    __syncwarp();
    int before = 0;
    if (lane == 0)
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;\n" : "=r"(before) : "l"(p.done + block) : "memory");
    if (__shfl_sync(0xffffffffu, before, 0) != parts - 1) return true;
    // the block's last warp merges all parts: a lane half of a row's, in order
    __syncwarp();
    const int r = lane % kWeighRows;
    float mm = -INFINITY, ll = 0.f;
    if (r < 8 * NB) {
#pragma unroll 8
        for (int k = lane / kWeighRows; k < parts; k += 2) {
            const float2 v = __ldcg(part + k * kWeighRows + r);
            join(mm, ll, v.x, v.y);
        }
    }
    join(mm, ll, __shfl_down_sync(0xffffffffu, mm, kWeighRows), __shfl_down_sync(0xffffffffu, ll, kWeighRows));
    if (lane < n_rows) {
        const int row = row0 + r, g = row - p.group.div(row) * p.G;
        ll = add_sink(ll, p.sinks, head0 + g, mm);
        // a row that sees nothing gives nothing
        p.stat[(size_t)block * kWeighRows + r] = mm == -INFINITY ? INFINITY : mm + log2f(ll);
    }
    return true;
}

template <int D, int KT>
__global__ void __launch_bounds__(kStatThreads, Ring<D, KT>::CTAS) rpa_weigh_stats_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                                          const WeighParams p) {
    using R = Ring<D, KT>;
    extern __shared__ uint8_t s_raw[];
    __shared__ __align__(8) uint64_t s_full[R::STAGES], s_empty[R::STAGES];
    __shared__ StageMeta meta[R::STAGES];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = (smem_u32(s_raw) + 127u) & ~127u, full = smem_u32(s_full), empty = smem_u32(s_empty);
    if (threadIdx.x == 0) {
        for (int i = 0; i < R::STAGES; ++i) {
            mbar_init(full + i * 8, 1);
            mbar_init(empty + i * 8, kConsumers);
        }
        fence_mbar_init();
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();
    int st = 0;
    uint32_t phase = 0;
    if (warp == kConsumers) {
        // ---- producer
        const int items = p.ctrl[0], BR = p.BR, runs = R::KEYS / BR;
        bool ok = true;
        int it = 0, nxt = 0;
        if (lane == 0) it = atomicAdd(p.ctrl + 2, 1);
        it = __shfl_sync(0xffffffffu, it, 0);
        while (ok && it < items) {
            if (lane == 0) nxt = atomicAdd(p.ctrl + 2, 1);
            // items of a sequence: piece, then row block, then kv head (neighbours read neighbouring rows)
            Piece c;
            c.s = find_seq(p.stat0, p.S, it, lane);
            c.q0 = p.cu[c.s];
            c.ql = p.cu[c.s + 1] - c.q0;
            c.kl = p.kv_lens[c.s];
            const int first = p.stat0[c.s], at = it - first;
            c.nb = (c.ql * p.G + kWeighRows - 1) / kWeighRows;
            c.pieces = (p.stat0[c.s + 1] - first) / (c.nb * p.Hkv);
            c.h = at % p.Hkv;
            c.rb = at / p.Hkv % c.nb;
            c.piece = at / p.Hkv / c.nb;
            cut(p, c);
            int k_first, k_last;
            seen(p, c, k_first, k_last);
            // K is read once where there is one row block: it leaves L2 to the logits
            const uint64_t policy = c.nb == 1 ? l2_policy_evict_first() : l2_policy_normal();
            const int* table = p.page_indices + (size_t)c.s * p.P;
            // lane r: page run r of a stage, its page id looked up a stage ahead
            auto look = [&](int k0) { return __ldg(table + p.page.div(min(k0 + lane * BR, max(k_last, 1) - 1))); };
            int page = look(k_first);
            int k0 = k_first;
            do {
                if (!mbar_wait(empty + st * 8, phase ^ 1u, p.status, kWeighWaitNs)) {
                    ok = false;
                    break;
                }
                const int k = k0 + lane * BR;
                const bool want = lane < runs && k < k_last, good = want && (unsigned)page < (unsigned)p.N;
                if (want && !good) set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
                const uint32_t mask = __ballot_sync(0xffffffffu, good);
                if (lane == 0) {
                    StageMeta& m = meta[st];
                    if (k0 == k_first) {
                        m.c = c;
                        m.k_first = k_first;
                        m.k_last = k_last;
                    }
                    m.k0 = k0;
                    m.runs = mask;
                    m.stop = 0;
                    mbar_arrive_expect_tx(full + st * 8, (uint32_t)__popc(mask) * (uint32_t)(BR * R::ROW));
                }
                __syncwarp();
                if (good)
                    tma_load_3d_hint(ring + st * R::STAGE + lane * (BR * R::ROW), &kmap, full + st * 8, 0,
                                     page * p.ps + (k - p.page.div(k) * p.ps), 2 * c.h * (R::ROW / 64), policy);
                if (++st == R::STAGES) {
                    st = 0;
                    phase ^= 1u;
                }
                k0 += R::KEYS;
                if (k0 < k_last) page = look(k0);
            } while (k0 < k_last);
            it = __shfl_sync(0xffffffffu, nxt, 0);
        }
        if (ok && mbar_wait(empty + st * 8, phase ^ 1u, p.status, kWeighWaitNs)) {
            if (lane == 0) {
                meta[st].stop = 1;
                mbar_arrive(full + st * 8);
            }
        } else {
            // gave up: let the copies already issued land before leaving
            for (int i = 0; i < R::STAGES; ++i) mbar_wait(full + i * 8, i < st ? phase : phase ^ 1u, p.status, kWeighWaitNs);
        }
        return;
    }
    // ---- consumers
    for (;;) {
        if (!mbar_wait(full + st * 8, phase, p.status, kWeighWaitNs)) return;
        if (meta[st].stop) return;
        const Piece& c = meta[st].c;
        const bool few = min(kWeighRows, c.ql * p.G - c.rb * kWeighRows) <= 8;
        const bool ok = few ? stat_item<D, KT, 1>(p, meta, ring, full, empty, warp, st, phase)
                            : stat_item<D, KT, 2>(p, meta, ring, full, empty, warp, st, phase);
        if (!ok) return;
    }
}

// ---------------------------------------------------------------- weigh
// Where key j's score of kv head h is (nullptr: on no page)
__device__ __forceinline__ float* score_at(const WeighParams& p, const int* table, int h, int j) {
    const int lp = p.page.div(j), pg = __ldg(table + lp);
    return (unsigned)pg < (unsigned)p.N ? p.scores + ((size_t)pg * p.Hkv + h) * p.ps + (j - lp * p.ps) : nullptr;
}
// the call's own keys start from 0; the others add (a page may be shared by sequences)
__device__ __forceinline__ void add_score(float* dst, bool fresh, float w) {
    if (dst == nullptr) return;
    if (fresh) *dst = w;
    else atomicAdd(dst, w);
}
// the same of four keys from k0 on, those of negative weight left out, in one operation of 16 bytes where it can be
__device__ __forceinline__ void add_scores4(float* dst, int k0, int pos0, const float (&w)[4]) {
    const bool all = w[0] >= 0.f && w[1] >= 0.f && w[2] >= 0.f && w[3] >= 0.f;
    if (all && k0 + 4 <= pos0) {
        asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"l"(dst), "f"(w[0]), "f"(w[1]), "f"(w[2]), "f"(w[3]) : "memory");
    } else if (all && k0 >= pos0) {
        *reinterpret_cast<float4*>(dst) = make_float4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (!(w[k] < 0.f)) add_score(dst + k, k0 + k >= pos0, w[k]);
    }
}

// Key tiles of 16 a warp holds while it goes through the rows: 32 registers of K (64 at D 256)
__host__ __device__ constexpr int weigh_tiles(int loads) { return loads >= 4 ? 1 : 4 / loads; }

template <int D, int KT>
__global__ void __launch_bounds__(kWeighThreads, D == 256 ? 2 : 4) rpa_weigh_kernel(const WeighParams p) {
    constexpr int kTiles = weigh_tiles(Deal<D, KT>::LOADS);
    pdl_trigger();
    pdl_wait();
    const int items = p.ctrl[1], heads = p.ctrl[3], lane = threadIdx.x & 31, quad = lane % 4;
    for (int it = blockIdx.x * kWarps + (threadIdx.x >> 5); it < items; it += gridDim.x * kWarps) {
        const int s = find_seq(p.item0, p.S, it, lane);
        const int q0 = p.cu[s], ql = p.cu[s + 1] - q0, kl = p.kv_lens[s], pos0 = kl - ql;
        const long long lo0 = p.logit0[s];
        const int hp = lo0 >= 0 ? heads : 1, groups = (p.Hkv + hp - 1) / hp;  // kv heads of an item
        const int base = first_key(p, kl, ql), at = it - p.item0[s], h = at % groups * hp;
        const int n_keys = lo0 >= 0 ? kWeighKeys : 16 * kTiles;
        const int j0 = base + at / groups * n_keys, j1 = min(kl, j0 + n_keys);
        const int lo = p.has_window ? max(0, pos0 - p.window + 1) : 0;  // keys below are seen by no row
        const int rows = ql * p.G, nb = (rows + kWeighRows - 1) / kWeighRows;
        const int* table = p.page_indices + (size_t)s * p.P;
        const float* stat = p.stat + (size_t)(p.block0[s] + h * nb) * kWeighRows;
        if (lo0 >= 0) {
            // four neighbouring keys a lane (of one page: page sizes are multiples of 4); lane r holds row r's statistic
            constexpr int KL = kWeighKeys / 32;
            static_assert(KL == 4, "add_scores4");
            const int rs = (rows + 1) & ~1, k0 = j0 + KL * lane;
            float* dst = k0 < j1 && k0 + KL > lo ? score_at(p, table, h, k0) : nullptr;
            const int h_end = min(p.Hkv, h + hp);
#pragma unroll 1
            for (int head = h; head < h_end; ++head, stat += kWeighRows) {
                const float st = lane < rows ? stat[lane] : 0.f;
                const float* x = p.logits + lo0 + (size_t)head * (kl - base) * rs;
                float w[KL];
                const float* xk[KL];
#pragma unroll
                for (int k = 0; k < KL; ++k) {
                    xk[k] = x + (size_t)(min(k0 + k, j1 - 1) - base) * rs;
                    w[k] = 0.f;
                }
                int r = 0;
                if (rs % 4 == 0) {
                    for (; r < rs; r += 4) {
                        float4 v[KL];
#pragma unroll
                        for (int k = 0; k < KL; ++k) v[k] = *reinterpret_cast<const float4*>(xk[k] + r);
                        // the place behind an odd number of rows is no row's (it holds the last one again)
                        if (r + 3 >= rows) {
#pragma unroll
                            for (int k = 0; k < KL; ++k) v[k].w = -INFINITY;
                        }
                        const float s0 = __shfl_sync(0xffffffffu, st, r), s1 = __shfl_sync(0xffffffffu, st, r + 1);
                        const float s2 = __shfl_sync(0xffffffffu, st, r + 2), s3 = __shfl_sync(0xffffffffu, st, r + 3);
#pragma unroll
                        for (int k = 0; k < KL; ++k)
                            w[k] += (ex2(v[k].x - s0) + ex2(v[k].y - s1)) + (ex2(v[k].z - s2) + ex2(v[k].w - s3));
                    }
                } else {
                    for (; r < rs; r += 2) {
                        float2 v[KL];
#pragma unroll
                        for (int k = 0; k < KL; ++k) v[k] = *reinterpret_cast<const float2*>(xk[k] + r);
                        if (r + 1 >= rows) {
#pragma unroll
                            for (int k = 0; k < KL; ++k) v[k].y = -INFINITY;
                        }
                        const float s0 = __shfl_sync(0xffffffffu, st, r), s1 = __shfl_sync(0xffffffffu, st, r + 1);
#pragma unroll
                        for (int k = 0; k < KL; ++k) w[k] += ex2(v[k].x - s0) + ex2(v[k].y - s1);
                    }
                }
#pragma unroll
                for (int k = 0; k < KL; ++k)
                    if (k0 + k < lo || k0 + k >= j1) w[k] = -1.f;
                if (dst) add_scores4(dst + (size_t)(head - h) * p.ps, k0, pos0, w);
            }
        } else {
            KeyTile<D, KT> t[kTiles];
            float w[kTiles][2];
            const uint64_t policy = l2_policy_normal();
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                load_k<D, KT>(p, table, h, j0 + 16 * i, j1, lane, policy, t[i]);
                w[i][0] = w[i][1] = 0.f;
            }
            bool full = true;  // every key of the tiles is there
#pragma unroll
            for (int i = 0; i < kTiles; ++i) full = full && t[i].ok[0] && t[i].ok[1];
            full = __all_sync(0xffffffffu, full);
            // rows whose tokens see one of the keys
            int r_lo = 0, r_hi = rows;
            if (p.causal) r_lo = max(0, j0 - pos0) * p.G & ~7;
            if (p.has_window) r_hi = (int)min((long long)rows, max(0ll, (long long)j1 - 1 + p.window - pos0) * p.G);
            // operands of kDeep row blocks: the loads of the next ones (an L2 latency of several blocks) behind this one
            constexpr int kDeep = D == 64 ? 4 : D == 128 && !kt_8bit(KT) ? 3 : 2;
            uint32_t q[kDeep][1][Deal<D, KT>::REGS];
            float2 st[kDeep];  // of rows 2 quad and 2 quad + 1
            auto fetch = [&](int r0, int b) {
                load_q<D, KT>(p, q0, h, r0 + lane / 4, rows, quad, q[b][0]);
                // rows behind the last weigh nothing
                st[b] = *reinterpret_cast<const float2*>(stat + r0 + 2 * quad);
                if (r0 + 2 * quad >= rows) st[b].x = INFINITY;
                if (r0 + 2 * quad + 1 >= rows) st[b].y = INFINITY;
            };
            auto add = [&](auto masked, int r0, int b) {
                constexpr bool MASK = decltype(masked)::value;
                const int r = r0 + 2 * quad;
                const int pa = MASK ? pos0 + p.group.div(r) : 0, pb = MASK ? pos0 + p.group.div(r + 1) : 0;
#pragma unroll
                for (int i = 0; i < kTiles; ++i) {
                    float acc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
                    tile_dot<D, KT, 1>(t[i], q[b], acc);
                    scale(p, acc[0]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = j0 + 16 * i + 8 * k + lane / 4;
                        w[i][k] += ex2(hide<MASK>(p, acc[0][2 * k], j, pa, t[i].ok[k]) - st[b].x) +
                                   ex2(hide<MASK>(p, acc[0][2 * k + 1], j, pb, t[i].ok[k]) - st[b].y);
                    }
                }
            };
            const bool seen_by_all = full && !p.has_window && (!p.causal || j0 + 16 * kTiles - 1 <= pos0);
            auto step = [&](int r0, int b) {
                if (seen_by_all) return add(std::false_type{}, r0, b);
                const int a = pos0 + p.group.div(r0), z = pos0 + p.group.div(min(r0 + 7, rows - 1));
                if (full && !some_hidden(p, j0, j0 + 16 * kTiles, a, z)) add(std::false_type{}, r0, b);
                else add(std::true_type{}, r0, b);
            };
#pragma unroll
            for (int b = 0; b + 1 < kDeep; ++b)
                if (r_lo + 8 * b < r_hi) fetch(r_lo + 8 * b, b);
            for (int r0 = r_lo; r0 < r_hi; r0 += 8 * kDeep) {
#pragma unroll
                for (int b = 0; b < kDeep; ++b) {
                    const int r = r0 + 8 * b;
                    if (r + 8 * (kDeep - 1) < r_hi) fetch(r + 8 * (kDeep - 1), (b + kDeep - 1) % kDeep);
                    if (r < r_hi) step(r, b);
                }
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    w[i][0] += __shfl_xor_sync(0xffffffffu, w[i][0], o);
                    w[i][1] += __shfl_xor_sync(0xffffffffu, w[i][1], o);
                }
                const int j = j0 + 16 * i + lane / 4 + 8 * quad;
                if (quad < 2 && j >= lo && j < j1) add_score(score_at(p, table, h, j), j >= pos0, quad ? w[i][1] : w[i][0]);
            }
        }
    }
}

template <int D, int KT>
struct WeighKern {
    static cudaError_t prepare(int* stats, int* weigh) {
        cudaError_t e = cudaFuncSetAttribute(rpa_weigh_stats_kernel<D, KT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D, KT>::SMEM);
        if (e == cudaSuccess)
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(stats, rpa_weigh_stats_kernel<D, KT>, kStatThreads, Ring<D, KT>::SMEM);
        return e != cudaSuccess ? e : cudaOccupancyMaxActiveBlocksPerMultiprocessor(weigh, rpa_weigh_kernel<D, KT>, kWeighThreads, 0);
    }
    static cudaError_t launch(const CUtensorMap& kmap, WeighParams p, int grid_weigh, cudaStream_t st) {
        p.weigh_warps = grid_weigh * kWarps;
        p.item_keys = 16 * weigh_tiles(Deal<D, KT>::LOADS);
        cudaError_t e = launch_pdl(rpa_weigh_plan_kernel, 1, kPlanThreads, 0, st, p);
        if (e == cudaSuccess) e = launch_pdl(rpa_weigh_stats_kernel<D, KT>, p.ctas, kStatThreads, Ring<D, KT>::SMEM, st, kmap, p);
        if (e == cudaSuccess) e = launch_pdl(rpa_weigh_kernel<D, KT>, grid_weigh, kWeighThreads, 0, st, p);
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

cudaError_t weigh_prepare(int D, int kt, int* stats, int* weigh) {
    return weigh_dispatch(D, kt, [&](auto k) { return decltype(k)::prepare(stats, weigh); });
}
cudaError_t launch_weigh(const CUtensorMap& kmap, const WeighParams& p, int kt, int grid_weigh, cudaStream_t st) {
    return weigh_dispatch(p.D, kt, [&](auto k) { return decltype(k)::launch(kmap, p, grid_weigh, st); });
}

}  // namespace rpa
