// rpa_evict.cu -- the choice of the keys a sequence keeps, the compaction of the cache, and the host
// side of the eviction handle (rpa_evict_*; the weights' kernels are in rpa_weigh.cu).
//
// Two launches:
//
//   select   a cluster of 1 to 4 CTAs per (sequence, kv head).  The keys between the protected first and
//            the recent last ones compete for the budget's other places: the k-th largest score by a radix
//            select over the scores as ordered integers (three digits of 11, 11 and 10 bits, a histogram in
//            shared memory each; the first digit holds the sign, the exponent and two bits of the mantissa,
//            so that scores of all sizes spread over its bins).  Each CTA keeps the scores of its share of
//            the keys in shared memory, and adds up all CTAs' histograms for itself through distributed
//            shared memory.  Then one ordered pass lists the kept slots: each warp lists a run of
//            neighbouring keys, so that one scan over the warps and CTAs gives every warp its place and its
//            share of the ties, which go to the lowest slots.  A digit whose bin is wanted whole is the last.  Bound by its rounds of waits (three digits,
//            a few microseconds each), so few units take large clusters, as long as two thirds of the SMs hold them.
//   move     K and V of a head are neighbours in a slot, a row is one copy of 2 D elements.  A CTA takes as
//            many rows a round as its registers hold (32 to 256: eight 16-byte vectors a thread), and looks
//            the next round's up beside the reads.  Bound by reading and writing those rows.  Onto fresh
//            pages all rounds are independent.  Where the new pages hold other kept rows (in place), a
//            head's rows move in ascending order: kept row i sits at slot j >= i and goes to slot i, so that
//            a row may be written once all rows up to it are read, and what is read later is never written
//            before.  A cluster of up to 8 CTAs takes a head and meets between reads and writes.
//
// Both launches are shaped by what the handle was made for (max_num_seqs, pages_per_seq), not by a call's num_seqs.
//
// 64 sequences of up to 8 k keys cut to 2 k (8 heads, D 128, bf16; 1.09 GB): 194 us, of which select 23 and move
// 170 (6.4 TB/s); in place 229.  Two of 100 k keys cut to 16 k (e4m3, 139 MB): 48 us, 23 and 25; in place 84 (16
// heads, one CTA each: 240; the lookups not ahead of the reads: 532).
#include <math.h>
#include <string.h>

#include <cmath>
#include <new>

#include "rpa_evict.cuh"

namespace rpa {

namespace {

constexpr int kBins = 2048;
constexpr int kMaxCluster = 4;
constexpr int kSelCached = 40 * 1024;  // scores a CTA keeps at most (160 KB); further ones are read again
constexpr int kMoveThreads = 256;
constexpr int kMoveCtas = 3;   // resident an SM onto fresh pages (64 x 8 k: 194 us; two 207; four 322, their vectors spilled)
constexpr int kPlaceCtas = 2;  // the same in place, where clusters are few
constexpr int kMaxMoveCluster = 8;

// A score as an integer of the same order; NaN lowest, -0 as +0
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;\n" ::: "memory");
}
// Words of CTA `rank`'s shared memory, at the place that `addr` has in this CTA's
__device__ __forceinline__ uint2 cluster_load2(uint32_t addr, uint32_t rank) {
    uint32_t at;
    uint2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(at) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}
// Exclusive sum of v over the block's threads before this one, and the total
template <int kSelWarps>
__device__ __forceinline__ uint32_t block_before(uint32_t v, uint32_t* s_warp, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t sum = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    uint32_t w = lane < kSelWarps ? s_warp[lane] : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const uint32_t before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return sum - v + (warp > 0 ? before : 0u);
}

// CLUSTER: several CTAs of 1024 threads a unit (few units: their own time counts), one an SM, for two on one SM would
// share its issue slots while others idle; else one of 512 (many units: three CTAs an SM)
template <bool CLUSTER>
__global__ void __launch_bounds__(CLUSTER ? 1024 : 512, CLUSTER ? 1 : 3) rpa_evict_select_kernel(const CompactParams p) {
    constexpr int kSelThreads = CLUSTER ? 1024 : 512, kSelWarps = kSelThreads / 32;
    extern __shared__ __align__(16) uint32_t s_key[];  // [cached] the scores of the first of this CTA's competing keys
    __shared__ __align__(16) uint32_t s_hist[2][kBins];
    __shared__ uint32_t s_warp[kSelWarps], s_warp2[kSelWarps];
    __shared__ __align__(8) uint32_t s_count[2];  // of this CTA: keys above the threshold, keys equal to it
    __shared__ uint32_t s_digit, s_left, s_all;
    __shared__ int s_order;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = CLUSTER ? p.cluster : 1, rank = CLUSTER ? (int)cluster_rank() : 0, unit = blockIdx.x / C;
    const int s = unit / p.Hkv, h = unit - s * p.Hkv;
    pdl_trigger();
    pdl_wait();
    const int n = p.kv_lens[s];
    const bool first = rank == 0 && h == 0;
    if (n < 0 || n > p.P * p.ps) {  // the whole cluster leaves
        if (tid == 0) {
            set_status(p.status, RPA_ERR_BAD_LENGTHS);
            if (first) p.seq_n[s] = -1;
        }
        return;
    }
    const int* table = p.page_indices + (size_t)s * p.P;
    const int kept = min(n, p.budget);
    int* list = p.list + ((size_t)s * p.Hkv + h) * p.budget;
    const int step = C * kSelThreads, me = rank * kSelThreads + tid;  // of the cluster's threads
    if (first) {
        // rows on pages that stay where they are move in order, unless those pages are protected whole or nothing moves
        if (tid == 0) s_order = 0;
        __syncthreads();
        if (n > p.budget) {
            const int from = p.protect / p.ps, pages = (kept + p.ps - 1) / p.ps;
            const int* to = p.new_pages + (size_t)s * p.P;
            for (int i = from + tid; i < pages; i += kSelThreads)
                if (table[i] == to[i]) s_order = 1;
        }
        __syncthreads();
        if (tid == 0) {
            p.seq_n[s] = kept;
            p.seq_order[s] = s_order;
        }
    }
    if (p.fill)
        for (int i = kept + me; i < p.budget; i += step) list[i] = -1;
    if (n <= p.budget) {
        for (int i = me; i < n; i += step) list[i] = i;
        return;
    }
    for (int i = me; i < p.protect; i += step) list[i] = i;
    for (int i = me; i < p.recent; i += step) list[p.budget - p.recent + i] = n - p.recent + i;
    const uint32_t k = (uint32_t)(p.budget - p.protect - p.recent);
    if (k == 0) return;
    // the competing keys [lo_key, hi_key), in quads of neighbouring slots (page sizes are multiples of 4); this CTA's
    // share is `mine` quads from quad q0 on, of which the first and the last may hold keys that do not compete
    const int lo_key = p.protect, hi_key = n - p.recent;
    const int quads = (hi_key + 3) / 4 - lo_key / 4, share = (quads + C - 1) / C;
    const int q0 = lo_key / 4 + min(quads, rank * share), mine = min(share, max(0, quads - rank * share));
    auto load = [&](int i) -> uint4 {  // quad i of this CTA's
        const int j = 4 * (q0 + i), lp = p.page.div(j), pg = __ldg(table + lp);
        if ((unsigned)pg >= (unsigned)p.N) {
            set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
            return make_uint4(0u, 0u, 0u, 0u);
        }
        const float4 x = *reinterpret_cast<const float4*>(p.scores + ((size_t)pg * p.Hkv + h) * p.ps + (j - lp * p.ps));
        return make_uint4(ordered(x.x), ordered(x.y), ordered(x.z), ordered(x.w));
    };
    uint4* s_quad = reinterpret_cast<uint4*>(s_key);
    const int cached = p.cached / 4;
    auto quad = [&](int i) { return i < cached ? s_quad[i] : load(i); };
    // bit e: element e of quad i competes
    auto inside = [&](int i) -> uint32_t {
        const int j = 4 * (q0 + i);
        uint32_t m = 15u;
        if (j < lo_key) m &= 15u << (lo_key - j);
        if (j + 4 > hi_key) m &= 15u >> (j + 4 - hi_key);
        return m;
    };
    // the first digit's histogram while the scores come in
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[0][i] = 0;
    __syncthreads();
    constexpr int kFly = 4;
    for (int i0 = tid; i0 < mine; i0 += kFly * kSelThreads) {
        uint4 u[kFly];
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int i = i0 + f * kSelThreads;
            if (i < mine) u[f] = load(i);
        }
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int i = i0 + f * kSelThreads;
            if (i < mine) {
                if (i < cached) s_quad[i] = u[f];
                const uint32_t in = inside(i);
                if (in & 1u) atomicAdd(&s_hist[0][u[f].x >> 21], 1u);
                if (in & 2u) atomicAdd(&s_hist[0][u[f].y >> 21], 1u);
                if (in & 4u) atomicAdd(&s_hist[0][u[f].z >> 21], 1u);
                if (in & 8u) atomicAdd(&s_hist[0][u[f].w >> 21], 1u);
            }
        }
    }
    // the k-th largest key: digit by digit, the prefix found so far and how many are still wanted at and below it
    uint32_t prefix = 0, left = k;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
        uint32_t* hist = s_hist[d & 1];
        if (d > 0) {
            // (every CTA has read this half's last histogram before the barrier of the digit in between)
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < mine; i += kSelThreads) {
                const uint4 u = quad(i);
                const uint32_t in = inside(i);
                auto count = [&](uint32_t v, uint32_t bit) {
                    if ((v >> (shift + bits)) == prefix && (in & bit)) atomicAdd(&hist[(v >> shift) & ((1u << bits) - 1)], 1u);
                };
                count(u.x, 1u);
                count(u.y, 2u);
                count(u.z, 4u);
                count(u.w, 8u);
            }
        }
        if (CLUSTER) cluster_sync();
        else __syncthreads();
        // thread t: the kMine bins from kBins - 1 - kMine t down, over all CTAs; c[0] the highest
        constexpr int kMine = kBins / kSelThreads;
        static_assert(kMine == (CLUSTER ? 2 : 4), "one load a CTA");
        const int low = kBins - kMine * (tid + 1);
        uint32_t c[kMine];
        if constexpr (CLUSTER) {
            uint2 x[kMaxCluster];  // all CTAs' loads in flight
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) x[r] = r < C ? cluster_load2(smem_u32(hist + low), r) : make_uint2(0u, 0u);
            c[0] = c[1] = 0;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                c[1] += x[r].x;
                c[0] += x[r].y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < kMine; ++i) c[i] = hist[low + kMine - 1 - i];
        }
        uint32_t mine_sum = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) mine_sum += c[i];
        uint32_t total, above = block_before<kSelWarps>(mine_sum, s_warp, total);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            if (above < left && left <= above + c[i]) {
                s_digit = (uint32_t)(low + kMine - 1 - i);
                s_left = left - above;
                s_all = left == above + c[i];  // every key of the bin
            }
            above += c[i];
        }
        __syncthreads();
        prefix = (prefix << bits) | s_digit;
        left = s_left;
        if (s_all && prefix != 0u) {  // the keys from `prefix` on and no ties: the threshold is below its lowest key
            prefix = (prefix << shift) - 1u;
            left = 0;
            break;
        }
        __syncthreads();  // s_digit, s_left and s_warp are free again
    }
    // list the kept slots in order: keys above the threshold and the first `left` that equal it
    const int run = ((mine + kSelWarps - 1) / kSelWarps + 31) & ~31, lo = min(mine, warp * run), hi = min(mine, lo + run);
    // of quad i: bits of the keys above the threshold, and 4 places up of those that equal it
    auto sift = [&](int i) -> uint32_t {
        const uint4 u = quad(i);
        const uint32_t in = inside(i);
        const uint32_t g = (u.x > prefix ? 1u : 0u) | (u.y > prefix ? 2u : 0u) | (u.z > prefix ? 4u : 0u) | (u.w > prefix ? 8u : 0u);
        const uint32_t e = (u.x == prefix ? 1u : 0u) | (u.y == prefix ? 2u : 0u) | (u.z == prefix ? 4u : 0u) | (u.w == prefix ? 8u : 0u);
        return (g & in) | (e & in) << 4;
    };
    uint32_t gt = 0, eq = 0;
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t m = sift(i);
        gt += __popc(m & 15u);
        eq += __popc(m >> 4);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    uint32_t all_gt, all_eq;
    uint32_t g0 = block_before<kSelWarps>(lane == 0 ? gt : 0u, s_warp, all_gt);
    uint32_t e0 = block_before<kSelWarps>(lane == 0 ? eq : 0u, s_warp2, all_eq);
    g0 = __shfl_sync(0xffffffffu, g0, 0);
    e0 = __shfl_sync(0xffffffffu, e0, 0);
    if constexpr (CLUSTER) {
        if (tid == 0) {
            s_count[0] = all_gt;
            s_count[1] = all_eq;
        }
        cluster_sync();
        const uint2 v = lane < rank ? cluster_load2(smem_u32(s_count), lane) : make_uint2(0u, 0u);  // lane r: CTA r
        g0 += __reduce_add_sync(0xffffffffu, v.x);
        e0 += __reduce_add_sync(0xffffffffu, v.y);
    }
    for (int i = lo; i < hi; i += 32) {
        const uint32_t m = i + lane < hi ? sift(i + lane) : 0u;
        // both counts of the lanes before this one in one scan (at most 128 each)
        const uint32_t own = __popc(m & 15u) | __popc(m >> 4) << 16;
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        uint32_t g = g0 + ((sum - own) & 0xffffu), e = e0 + ((sum - own) >> 16);
        const uint32_t all = __shfl_sync(0xffffffffu, sum, 31);
        g0 += all & 0xffffu;
        e0 += all >> 16;
        if (m == 0u) continue;
        int* out = list + p.protect;
        const int j = 4 * (q0 + i + lane);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            if (m >> x & 1u) {
                out[g + min(e, left)] = j + x;
                ++g;
            } else if (m >> (4 + x) & 1u) {
                if (e < left) out[g + e] = j + x;
                ++e;
            }
        }
    }
    if (CLUSTER) cluster_sync();  // no CTA leaves while another may read its counts
}

// Kept row i of head h: where it is and where it goes (first 16-byte vectors; to -1: it stays, or has no page), and its score's
// new place (nullptr: none) and value
struct Row {
    long long from, to;
    float* sc_to;
    float sc;
};
__device__ __forceinline__ Row look_up(const CompactParams& p, int s, int h, int i, int j) {
    Row r = {0, -1, nullptr, 0.f};
    const int pj = p.page.div(j), pi = p.page.div(i);
    const int pa = __ldg(p.page_indices + (size_t)s * p.P + pj), pb = __ldg(p.new_pages + (size_t)s * p.P + pi);
    if ((unsigned)pa >= (unsigned)p.N || (unsigned)pb >= (unsigned)p.N) {
        set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
        return r;
    }
    const int at = j - pj * p.ps, bt = i - pi * p.ps;
    r.from = (((long long)pa * p.ps + at) * p.Hkv + h) << p.vec_shift;
    const long long to = (((long long)pb * p.ps + bt) * p.Hkv + h) << p.vec_shift;
    if (to != r.from) {
        r.to = to;
        r.sc = p.scores[((size_t)pa * p.Hkv + h) * p.ps + at];
        r.sc_to = p.scores + ((size_t)pb * p.Hkv + h) * p.ps + bt;
    }
    return r;
}

constexpr int kFly = 8;  // 16-byte vectors a thread has in flight

// Rounds of rows, as many as the CTA's registers hold: read, meet (with the CTAs of a cluster), write.  where(n) is this
// thread's row of round n, looked up a round ahead, beside the reads.
template <bool CLUSTER, typename Where>
__device__ __forceinline__ void move_rounds(const CompactParams& p, int rounds, long long (*s_from)[kMoveThreads],
                                            long long (*s_to)[kMoveThreads], Where where) {
    uint4* kv = reinterpret_cast<uint4*>(p.kv);
    const int tid = threadIdx.x, vecs = 1 << p.vec_shift;  // 16-byte vectors of a row: 8, 16, 32 or 64
    Row row = where(0);
    __syncthreads();  // the tables' last round
    s_from[0][tid] = row.from;
    s_to[0][tid] = row.to;
    __syncthreads();
    int at = 0;  // the round's third of the tables
    for (int n = 0; n < rounds; ++n) {
        const int next = at == 2 ? 0 : at + 1;
        uint4 x[kFly];
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int v = tid + f * kMoveThreads, r = v >> p.vec_shift;
            if (s_to[at][r] >= 0) x[f] = __ldcs(kv + s_from[at][r] + (v & (vecs - 1)));
        }
        const Row ahead = where(n + 1);
        s_from[next][tid] = ahead.from;
        s_to[next][tid] = ahead.to;
        if (CLUSTER) cluster_sync();
        else __syncthreads();
#pragma unroll
        for (int f = 0; f < kFly; ++f) {
            const int v = tid + f * kMoveThreads, r = v >> p.vec_shift;
            if (s_to[at][r] >= 0) __stcs(kv + s_to[at][r] + (v & (vecs - 1)), x[f]);
        }
        if (row.sc_to) *row.sc_to = row.sc;
        row = ahead;
        at = next;
    }
}

// IN_PLACE: the new pages are the old ones, rows move in order or not at all, a cluster a head.  Else each sequence by its own rule
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveThreads, IN_PLACE ? kPlaceCtas : kMoveCtas) rpa_evict_move_kernel(const CompactParams p) {
    __shared__ long long s_from[3][kMoveThreads], s_to[3][kMoveThreads];  // Row::from and to
    const int tid = threadIdx.x, per_cta = kFly * kMoveThreads >> p.vec_shift;  // rows of a CTA's round
    pdl_trigger();
    pdl_wait();
    const int units = p.S * p.Hkv, C = IN_PLACE ? p.move_cluster : 1, rank = IN_PLACE ? (int)cluster_rank() : 0;
    for (int u = blockIdx.x / C; u < units; u += gridDim.x / C) {
        const int s = u / p.Hkv, h = u - s * p.Hkv, kept = p.seq_n[s];
        if (IN_PLACE && kept >= 0 && h == 0 && rank == 0 && tid == 0) p.new_kv_lens[s] = kept;
        if (kept <= 0 || p.seq_order[s] == 0) continue;
        // all kept rows of a head onto pages that hold others of them; a row's slot is read two rounds ahead
        const int* list = p.list + ((size_t)s * p.Hkv + h) * p.budget;
        const int step = C * per_cta, mine = rank * per_cta + tid;
        auto slot = [&](int n) { return tid < per_cta && (long long)n * step + mine < kept ? list[n * step + mine] : -1; };
        int j = slot(0);
        move_rounds<IN_PLACE>(p, (kept + step - 1) / step, s_from, s_to, [&](int n) {
            Row r = {0, -1, nullptr, 0.f};
            if (j >= 0) r = look_up(p, s, h, n * step + mine, j);
            j = slot(n + 1);
            return r;
        });
    }
    if (IN_PLACE) return;
    // onto fresh pages: blocks of rows in any order
    const int blocks = (p.budget + per_cta - 1) / per_cta, items = units * blocks;
    const int rounds = (items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
    move_rounds<false>(p, rounds, s_from, s_to, [&](int n) {
        Row r = {0, -1, nullptr, 0.f};
        if (n >= rounds) return r;
        const int it = blockIdx.x + n * gridDim.x, h = it % p.Hkv, b = it / p.Hkv % blocks, s = it / p.Hkv / blocks;
        const int kept = p.seq_n[s], i = b * per_cta + tid;
        if (b == 0 && h == 0 && tid == 0 && kept >= 0) p.new_kv_lens[s] = kept;
        if (tid < per_cta && i < kept && p.seq_order[s] == 0) r = look_up(p, s, h, i, p.list[((size_t)s * p.Hkv + h) * p.budget + i]);
        return r;
    });
}

}  // namespace

// Clusters and shared memory of select for `units` (sequence, kv head) pairs of up to max_keys competing keys
cudaError_t compact_prepare(int64_t units, int max_keys, int sms, int* cluster, int* move_cluster, int* cached) {
    // as many CTAs a unit as two thirds of the SMs hold, one each, with 2 k keys at least
    int c = 1;
    while (c < kMaxCluster && 3 * units * (2 * c) <= 2 * sms && max_keys / (2 * c) >= 2048) c *= 2;
    *cluster = c;
    // rows that move in order: as many CTAs a unit as there are
    int m = 1;
    while (m < kMaxMoveCluster && units * (2 * m) <= sms * kPlaceCtas) m *= 2;
    *move_cluster = m;
    const int share = ((max_keys + 3) / 4 + 1 + c - 1) / c * 4;  // (one quad more where neither end is a quad's)
    *cached = share < kSelCached ? share : kSelCached;
    return cudaFuncSetAttribute(c > 1 ? rpa_evict_select_kernel<true> : rpa_evict_select_kernel<false>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCached * 4);
}

cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t st) {
    if (p.S == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.S * p.Hkv * p.cluster);
    cfg.blockDim = dim3(p.cluster > 1 ? 1024 : 512);
    cfg.dynamicSmemBytes = (size_t)p.cached * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, p.cluster > 1 ? rpa_evict_select_kernel<true> : rpa_evict_select_kernel<false>, p);
    if (e != cudaSuccess) return e;
    if (p.new_pages != p.page_indices) return launch_pdl(rpa_evict_move_kernel<false>, sms * kMoveCtas, kMoveThreads, 0, st, p);
    const int m = p.move_cluster;
    cfg.gridDim = dim3(p.S * p.Hkv * m);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    attr[1].val.clusterDim.x = m;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, rpa_evict_move_kernel<true>, p);
}

}  // namespace rpa

using namespace rpa;

struct RpaEvict {
    RpaEvictCfg cfg;
    int device, sms;
    KernelSet ks;      // element types and scales of the attention of `cfg.cache`
    int stats_bps, weigh_bps;  // resident CTAs an SM of the two weight kernels
    int cluster, cached;  // of select
    int move_cluster;
    void* ws;
    int* status;
    WeighParams w;     // workspace pointers and constants
    uint8_t* qbuf;     // q in the MMA operand type, where that is another
    int* list;
    int *seq_n, *seq_order;
};

namespace {

constexpr long long kMostLogits = 1ll << 28;  // floats: 1 GiB
constexpr int kMostPieces = 128;

}  // namespace

extern "C" {

int rpa_evict_validate_cfg(const RpaEvictCfg* c) {
    if (!c) return RPA_ERR_INVALID_ARG;
    const int v = rpa_validate_cfg(&c->cache);
    if (v != RPA_OK) return v;
    if (c->reserved != 0) return RPA_ERR_INVALID_ARG;
    if (c->budget < 1 || c->budget > c->cache.pages_per_seq * c->cache.page_size) return RPA_ERR_INVALID_ARG;
    if (c->protect < 0 || c->recent < 0 || c->protect > c->budget || c->recent > c->budget - c->protect)
        return RPA_ERR_INVALID_ARG;
    if (c->cache.kv_layout != RPA_KV_SPLIT || c->cache.first_keys > 0 || int4_group(c->cache.kv_dtype)) return RPA_ERR_UNSUPPORTED;
    // 32-bit numbers of keys (with room for sums of two), rows, slots, grids' CTAs and blocks of kept keys
    if (c->cache.pages_per_seq * c->cache.page_size > (int64_t)1 << 30) return RPA_ERR_UNSUPPORTED;
    const int64_t lim = (int64_t)1 << 31, units = c->cache.max_num_seqs * c->cache.num_kv_heads;
    if (c->cache.num_q_tokens * (c->cache.num_q_heads / c->cache.num_kv_heads) >= lim ||
        c->cache.total_num_pages >= lim / c->cache.page_size || units >= lim / 8 ||
        units >= lim / 4 / (c->budget / (kFly * kMoveThreads / 64) + 1))
        return RPA_ERR_UNSUPPORTED;
    return RPA_OK;
}

int rpa_evict_create(const RpaEvictCfg* cfg, RpaEvict** out) {
    if (!out) return RPA_ERR_INVALID_ARG;
    *out = nullptr;
    const int v = rpa_evict_validate_cfg(cfg);
    if (v != RPA_OK) return v;
    RpaEvict* h = new (std::nothrow) RpaEvict;
    if (!h) return RPA_ERR_CUDA;
    memset(h, 0, sizeof *h);
    h->cfg = *cfg;
    const RpaCfg& c = h->cfg.cache;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&h->sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return RPA_ERR_CUDA;
    }
    kernels_choose(c, h->sms, &h->ks);
    const int64_t max_keys = c.pages_per_seq * c.page_size;
    if (weigh_prepare(h->ks.D, h->ks.kt, &h->stats_bps, &h->weigh_bps) != cudaSuccess || h->stats_bps < 1 || h->weigh_bps < 1 ||
        compact_prepare(c.max_num_seqs * c.num_kv_heads, (int)max_keys, h->sms, &h->cluster, &h->move_cluster, &h->cached) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return RPA_ERR_CUDA;
    }
    // worst cases: row blocks (each sequence's last may be part empty), pieces, logits of sequences of one block
    const int64_t S = c.max_num_seqs, Hkv = c.num_kv_heads, rows = c.num_q_tokens * h->ks.G;
    const int64_t blocks = (rows / kWeighRows + S) * Hkv;
    int64_t pieces = ((int64_t)1 << 20) / blocks;
    pieces = pieces < 1 ? 1 : pieces > kMostPieces ? kMostPieces : pieces;
    const int64_t small_rows = rows + S < S * kWeighRows ? rows + S : S * kWeighRows;
    double most = (double)small_rows * (double)Hkv * (double)max_keys + 4.0 * (double)S;
    if (most > (double)kMostLogits) most = (double)kMostLogits;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t o_status = take(4), o_ctrl = take(16), o_stat0 = take((S + 1) * 4), o_item0 = take((S + 1) * 4),
                 o_block0 = take((S + 1) * 4), o_logit0 = take(S * 8), o_done = take(blocks * 4),
                 o_part = take((size_t)blocks * pieces * 4 * kWeighRows * 8), o_stat = take((size_t)blocks * kWeighRows * 4),
                 o_logits = take((size_t)most * 4), o_n = take(S * 4), o_order = take(S * 4),
                 o_list = take((size_t)S * Hkv * cfg->budget * 4),
                 o_q = take(h->ks.q_conv ? (size_t)c.num_q_tokens * c.num_q_heads * c.head_dim * 2 : 0);
    if (cudaMalloc(&h->ws, off) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return RPA_ERR_CUDA;
    }
    if (!set_now(cudaMemset(h->ws, 0, 256))) {
        cudaGetLastError();
        cudaFree(h->ws);
        delete h;
        return RPA_ERR_CUDA;
    }
    uint8_t* b = static_cast<uint8_t*>(h->ws);
    h->status = reinterpret_cast<int*>(b + o_status);
    h->qbuf = b + o_q;
    h->list = reinterpret_cast<int*>(b + o_list);
    h->seq_n = reinterpret_cast<int*>(b + o_n);
    h->seq_order = reinterpret_cast<int*>(b + o_order);
    WeighParams& w = h->w;
    w.T = (int)c.num_q_tokens;
    w.Hq = (int)c.num_q_heads;
    w.Hkv = (int)Hkv;
    w.G = h->ks.G;
    w.D = h->ks.D;
    w.ps = (int)c.page_size;
    w.P = (int)c.pages_per_seq;
    w.N = (int)c.total_num_pages;
    w.causal = c.is_causal ? 1 : 0;
    w.has_window = c.has_sliding_window ? 1 : 0;
    w.window = h->ks.window;
    w.has_cap = c.has_soft_cap ? 1 : 0;
    w.q_bf16 = kt_8bit(h->ks.kt) && !h->ks.q_f16;
    w.qk_log2 = h->ks.qk_log2;
    w.cap_arg = c.has_soft_cap ? (float)((double)c.sm_scale * (c.has_k_scale ? c.k_scale : 1.f) / c.soft_cap) : 0.f;
    w.cap_log2 = h->ks.cap_log2;
    w.sinks = c.has_sinks ? c.sinks : nullptr;
    w.page.set((uint32_t)w.ps);
    w.group.set((uint32_t)w.G);
    w.max_pieces = (int)pieces;
    w.ctas = h->sms * h->stats_bps;
    w.BR = h->ks.BR;
    w.br_shift = h->ks.br_shift;
    w.all_runs = (1u << (64 / w.BR)) - 1u;
    w.max_logits = (long long)most;
    w.status = h->status;
    w.ctrl = reinterpret_cast<int*>(b + o_ctrl);
    w.stat0 = reinterpret_cast<int*>(b + o_stat0);
    w.item0 = reinterpret_cast<int*>(b + o_item0);
    w.block0 = reinterpret_cast<int*>(b + o_block0);
    w.logit0 = reinterpret_cast<long long*>(b + o_logit0);
    w.done = reinterpret_cast<int*>(b + o_done);
    w.part = reinterpret_cast<float2*>(b + o_part);
    w.stat = reinterpret_cast<float*>(b + o_stat);
    w.logits = reinterpret_cast<float*>(b + o_logits);
    *out = h;
    return RPA_OK;
}

int rpa_evict_accumulate(RpaEvict* h, const void* q, const void* kv_pages, const int32_t* kv_lens,
                         const int32_t* page_indices, const int32_t* cu_q_lens, int32_t num_seqs, float* scores,
                         void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    const RpaCfg& c = h->cfg.cache;
    if (num_seqs < 0 || num_seqs > c.max_num_seqs) return RPA_ERR_INVALID_ARG;
    if (!kv_pages || !kv_lens || !page_indices || !cu_q_lens || !scores) return RPA_ERR_INVALID_ARG;
    if (c.num_q_tokens > 0 && !q) return RPA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(kv_pages, 16) || !aligned(kv_lens, 4) || !aligned(page_indices, 4) ||
        !aligned(cu_q_lens, 4) || !aligned(scores, 16))
        return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok) return RPA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    WeighParams p = h->w;
    p.q = static_cast<const uint8_t*>(q);
    p.kv = static_cast<const uint8_t*>(kv_pages);
    p.kv_lens = kv_lens;
    p.page_indices = page_indices;
    p.cu = cu_q_lens;
    p.scores = scores;
    p.S = num_seqs;
    if (h->ks.q_conv && c.num_q_tokens > 0) {
        const size_t n = (size_t)c.num_q_tokens * c.num_q_heads * c.head_dim;
        if (launch_q_convert(q, c.q_dtype, h->qbuf, h->ks.q_conv_f16, n, Launch{h->sms * 4, st}) != cudaSuccess) {
            cudaGetLastError();
            return RPA_ERR_CUDA;
        }
        p.q = h->qbuf;
    }
    CUtensorMap kmap;
    if (encode_k_map(&kmap, kv_pages, p.D * (kt_8bit(h->ks.kt) ? 1 : 2), c.total_num_pages, p.ps, p.Hkv, p.BR) != 0)
        return RPA_ERR_INVALID_ARG;
    if (launch_weigh(kmap, p, h->ks.kt, h->sms * h->weigh_bps, st) != cudaSuccess) {
        cudaGetLastError();
        return RPA_ERR_CUDA;
    }
    return RPA_OK;
}

int rpa_evict_compact(RpaEvict* h, void* kv_pages, float* scores, const int32_t* kv_lens, const int32_t* page_indices,
                      int32_t num_seqs, const int32_t* new_page_indices, int32_t* new_kv_lens, int32_t* kept,
                      void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    const RpaCfg& c = h->cfg.cache;
    if (num_seqs < 0 || num_seqs > c.max_num_seqs) return RPA_ERR_INVALID_ARG;
    if (!kv_pages || !scores || !kv_lens || !page_indices || !new_page_indices || !new_kv_lens) return RPA_ERR_INVALID_ARG;
    if (!aligned(kv_pages, 16) || !aligned(scores, 16) || !aligned(kv_lens, 4) || !aligned(page_indices, 4) ||
        !aligned(new_page_indices, 4) || !aligned(new_kv_lens, 4) || !aligned(kept, 4))
        return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok) return RPA_ERR_CUDA;
    CompactParams p;
    p.kv = static_cast<uint8_t*>(kv_pages);
    p.scores = scores;
    p.kv_lens = kv_lens;
    p.page_indices = page_indices;
    p.new_pages = new_page_indices;
    p.new_kv_lens = new_kv_lens;
    p.list = kept ? kept : h->list;
    p.fill = kept != nullptr;
    p.seq_n = h->seq_n;
    p.seq_order = h->seq_order;
    p.status = h->status;
    p.S = num_seqs;
    p.Hkv = (int)c.num_kv_heads;
    p.ps = (int)c.page_size;
    p.P = (int)c.pages_per_seq;
    p.N = (int)c.total_num_pages;
    const int vecs = (int)(2 * c.head_dim * (kt_8bit(h->ks.kt) ? 1 : 2) / 16);
    p.vec_shift = 0;
    while (1 << p.vec_shift < vecs) ++p.vec_shift;
    p.budget = (int)h->cfg.budget;
    p.protect = (int)h->cfg.protect;
    p.recent = (int)h->cfg.recent;
    p.cluster = h->cluster;
    p.move_cluster = h->move_cluster;
    p.cached = h->cached;
    p.page.set((uint32_t)p.ps);
    if (launch_compact(p, h->sms, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        cudaGetLastError();
        return RPA_ERR_CUDA;
    }
    return RPA_OK;
}

int rpa_evict_get_status(RpaEvict* h, void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    return g.ok ? take_status(h->status, static_cast<cudaStream_t>(stream)) : RPA_ERR_CUDA;
}

void rpa_evict_destroy(RpaEvict* h) {
    if (!h) return;
    DeviceGuard g(h->device);
    cudaFree(h->ws);
    delete h;
}

}  // extern "C"
