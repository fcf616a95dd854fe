// rpa_evict.cu -- the choice of the keys a sequence keeps, the compaction of the cache, and the host
// side of the eviction handle (rpa_evict_*; the weights' kernels are in rpa_weigh.cu).
//
// Two launches:
//
//   select   a CTA per (sequence, kv head).  The keys between the protected first and the recent last
//            ones compete for the budget's other places: the k-th largest score by a radix select over
//            the scores as ordered integers (three digits of 11, 11 and 10 bits, a shared-memory
//            histogram each: the first digit holds the sign, the exponent and two bits of the mantissa,
//            so that scores of all sizes spread over its bins), then one ordered pass that lists the
//            kept slots.  Each warp lists a run of neighbouring keys, so that one scan over the warps
//            gives every warp its place and its share of the ties, which go to the lowest slots.
//   move     blocks of 64 kept rows: K and V of a head are neighbours in a slot, one copy of 2 D
//            elements a row.  Bound by reading and writing those rows.  Onto fresh pages all blocks are
//            independent.  Where the new pages hold other kept rows (in place), a sequence's head is
//            done by one CTA in ascending order, a block read before it is written: kept row i sits at
//            slot j >= i and goes to slot i, so that a block's writes never reach a later block's rows.
#include <math.h>
#include <string.h>

#include <cmath>
#include <new>

#include "rpa_evict.cuh"

namespace rpa {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;

// A score as an integer of the same order; NaN lowest, -0 as +0
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) rpa_evict_select_kernel(const CompactParams p) {
    extern __shared__ uint32_t s_key[];  // [cached] the first competing keys' scores
    __shared__ uint32_t s_hist[kBins];
    __shared__ uint32_t s_warp[kSelWarps][2];
    __shared__ uint32_t s_digit, s_left;
    __shared__ int s_order;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.x / p.Hkv, h = blockIdx.x - s * p.Hkv;
    pdl_trigger();
    pdl_wait();
    const int n = p.kv_lens[s];
    if (n < 0 || n > p.P * p.ps) {
        if (tid == 0) {
            set_status(p.status, RPA_ERR_BAD_LENGTHS);
            if (h == 0) p.seq_n[s] = -1;
        }
        return;
    }
    const int* table = p.page_indices + (size_t)s * p.P;
    const int kept = min(n, p.budget);
    int* list = p.list + ((size_t)s * p.Hkv + h) * p.budget;
    if (h == 0) {
        // rows on pages that stay where they are: in order, unless those pages are protected whole or nothing moves
        if (tid == 0) s_order = 0;
        __syncthreads();
        if (n > p.budget) {
            const int first = p.protect / p.ps, pages = (kept + p.ps - 1) / p.ps;
            const int* to = p.new_pages + (size_t)s * p.P;
            for (int i = first + tid; i < pages; i += kSelThreads)
                if (table[i] == to[i]) s_order = 1;
        }
        __syncthreads();
        if (tid == 0) {
            p.seq_n[s] = kept;
            p.seq_order[s] = s_order;
        }
    }
    if (p.fill)
        for (int i = kept + tid; i < p.budget; i += kSelThreads) list[i] = -1;
    if (n <= p.budget) {
        for (int i = tid; i < n; i += kSelThreads) list[i] = i;
        return;
    }
    // the competing keys [protect, protect + m) and their places
    const int m = n - p.protect - p.recent;
    const uint32_t k = (uint32_t)(p.budget - p.protect - p.recent);
    auto score = [&](int i) -> uint32_t {  // of competing key i
        const int j = p.protect + i, lp = p.page.div(j), pg = __ldg(table + lp);
        if ((unsigned)pg >= (unsigned)p.N) {
            set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
            return 0u;
        }
        return ordered(p.scores[((size_t)pg * p.Hkv + h) * p.ps + (j - lp * p.ps)]);
    };
    auto key = [&](int i) { return i < p.cached ? s_key[i] : score(i); };
    for (int i = tid; i < min(m, p.cached); i += kSelThreads) s_key[i] = score(i);
    // the k-th largest key: digit by digit, the prefix found so far and how many are still wanted below it
    uint32_t prefix = 0, left = k;
    if (k > 0) {
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
            for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < m; i += kSelThreads) {
                const uint32_t u = key(i);
                if (d == 0 || (u >> (shift + bits)) == prefix) atomicAdd(&s_hist[(u >> shift) & ((1u << bits) - 1)], 1u);
            }
            __syncthreads();
            // thread t: bins kBins - 1 - 2t and the one below; an inclusive scan from the highest bin down
            const int b0 = kBins - 1 - 2 * tid;
            const uint32_t c0 = s_hist[b0], c1 = s_hist[b0 - 1];
            uint32_t sum = c0 + c1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            if (lane == 31) s_warp[warp][0] = sum;
            __syncthreads();
            uint32_t before = 0;
            for (int w = 0; w < warp; ++w) before += s_warp[w][0];
            const uint32_t above = before + sum - c0 - c1;  // keys in higher bins
            if (above < left && left <= above + c0) {
                s_digit = (uint32_t)b0;
                s_left = left - above;
            } else if (above + c0 < left && left <= above + c0 + c1) {
                s_digit = (uint32_t)b0 - 1;
                s_left = left - above - c0;
            }
            __syncthreads();
            prefix = (prefix << bits) | s_digit;
            left = s_left;
        }
    } else {
        prefix = 0xffffffffu;  // above every score: none competes
    }
    // list the kept slots in order: protected, keys above the threshold and the first `left` that equal it, recent
    for (int i = tid; i < p.protect; i += kSelThreads) list[i] = i;
    for (int i = tid; i < p.recent; i += kSelThreads) list[p.budget - p.recent + i] = n - p.recent + i;
    const int run = ((m + kSelWarps - 1) / kSelWarps + 31) & ~31, lo = min(m, warp * run), hi = min(m, lo + run);
    uint32_t gt = 0, eq = 0;
    __syncthreads();
    for (int i = lo + lane; i < hi; i += 32) {
        const uint32_t u = key(i);
        gt += u > prefix;
        eq += u == prefix;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        s_warp[warp][0] = gt;
        s_warp[warp][1] = eq;
    }
    __syncthreads();
    uint32_t g0 = 0, e0 = 0;
    for (int w = 0; w < warp; ++w) {
        g0 += s_warp[w][0];
        e0 += s_warp[w][1];
    }
    if (k == 0) return;
    for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi;
        const uint32_t u = in ? key(i + lane) : 0u;
        const uint32_t mg = __ballot_sync(0xffffffffu, in && u > prefix), me = __ballot_sync(0xffffffffu, in && u == prefix);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t e = e0 + __popc(me & below);
        if (in && (u > prefix || (u == prefix && e < left)))
            list[p.protect + g0 + __popc(mg & below) + min(e, left)] = p.protect + i + lane;
        g0 += __popc(mg);
        e0 += __popc(me);
    }
}

// Where kept row i of (s, h) comes from and goes to: slots of the cache (page * page_size + place), -1: no move
__device__ __forceinline__ void route(const CompactParams& p, int s, int h, int i, const int* list, long long& from, long long& to) {
    const int j = list[i];
    const int a = p.page.div(j), b = p.page.div(i);
    const int pa = __ldg(p.page_indices + (size_t)s * p.P + a), pb = __ldg(p.new_pages + (size_t)s * p.P + b);
    from = (long long)pa * p.ps + (j - a * p.ps);
    to = (long long)pb * p.ps + (i - b * p.ps);
    if ((unsigned)pa >= (unsigned)p.N || (unsigned)pb >= (unsigned)p.N) {
        set_status(p.status, RPA_ERR_BAD_PAGE_INDEX);
        to = -1;
    }
    if (from == to) to = -1;
}

__global__ void __launch_bounds__(kMoveThreads) rpa_evict_move_kernel(const CompactParams p) {
    __shared__ long long s_from[kMoveRows], s_to[kMoveRows];
    const int tid = threadIdx.x;
    pdl_trigger();
    pdl_wait();
    const int blocks = (p.budget + kMoveRows - 1) / kMoveRows;
    const long long items = (long long)p.S * p.Hkv * blocks;
    const int vecs = p.row_bytes / 16;  // 16-byte vectors of a row: 8, 16, 32 or 64
    const int slot_vecs = vecs * p.Hkv;
    uint4* kv = reinterpret_cast<uint4*>(p.kv);
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int h = (int)(it % p.Hkv), b = (int)(it / p.Hkv % blocks), s = (int)(it / p.Hkv / blocks);
        const int kept = p.seq_n[s];
        if (kept < 0) continue;
        if (b == 0 && h == 0 && tid == 0) p.new_kv_lens[s] = kept;
        const bool order = p.seq_order[s] != 0;
        if (order && b > 0) continue;
        const int* list = p.list + ((size_t)s * p.Hkv + h) * p.budget;
        const int end = order ? kept : min(kept, (b + 1) * kMoveRows);
        for (int i0 = b * kMoveRows; i0 < end; i0 += kMoveRows) {
            const int rows = min(kMoveRows, end - i0);
            float sc = 0.f;
            __syncthreads();
            if (tid < kMoveRows) {
                long long from = 0, to = -1;
                if (tid < rows) route(p, s, h, i0 + tid, list, from, to);
                s_from[tid] = from;
                s_to[tid] = to;
                if (to >= 0) {
                    const long long a = from / p.ps;
                    sc = p.scores[((size_t)a * p.Hkv + h) * p.ps + (from - a * p.ps)];
                }
            }
            __syncthreads();
            // 64 rows of up to 64 vectors: 16 a thread at most, eight in flight
            constexpr int kFly = 8;
            const int total = rows * vecs;
            if (!order) {
                for (int v0 = tid; v0 < total; v0 += kFly * kMoveThreads) {
                    uint4 x[kFly];
#pragma unroll
                    for (int f = 0; f < kFly; ++f) {
                        const int v = v0 + f * kMoveThreads, r = v / vecs;
                        if (v < total && s_to[r] >= 0) x[f] = kv[(size_t)s_from[r] * slot_vecs + h * vecs + (v - r * vecs)];
                    }
#pragma unroll
                    for (int f = 0; f < kFly; ++f) {
                        const int v = v0 + f * kMoveThreads, r = v / vecs;
                        if (v < total && s_to[r] >= 0) kv[(size_t)s_to[r] * slot_vecs + h * vecs + (v - r * vecs)] = x[f];
                    }
                }
            } else {
                // the whole block is read before any of it is written
                uint4 x[2 * kFly];
#pragma unroll
                for (int f = 0; f < 2 * kFly; ++f) {
                    const int v = tid + f * kMoveThreads, r = v / vecs;
                    if (v < total && s_to[r] >= 0) x[f] = kv[(size_t)s_from[r] * slot_vecs + h * vecs + (v - r * vecs)];
                }
                __syncthreads();
#pragma unroll
                for (int f = 0; f < 2 * kFly; ++f) {
                    const int v = tid + f * kMoveThreads, r = v / vecs;
                    if (v < total && s_to[r] >= 0) kv[(size_t)s_to[r] * slot_vecs + h * vecs + (v - r * vecs)] = x[f];
                }
            }
            if (tid < rows && s_to[tid] >= 0) {
                const long long a = s_to[tid] / p.ps;
                p.scores[((size_t)a * p.Hkv + h) * p.ps + (s_to[tid] - a * p.ps)] = sc;
            }
        }
    }
}

}  // namespace

// Shared memory of select: the scores of up to max_keys competing keys, as many as fit (40 k)
cudaError_t compact_prepare(int max_keys, int* cached) {
    *cached = max_keys < 40 * 1024 ? max_keys : 40 * 1024;
    return cudaFuncSetAttribute(rpa_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 40 * 1024 * 4);
}

cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t st) {
    if (p.S == 0) return cudaSuccess;
    cudaError_t e = launch_pdl(rpa_evict_select_kernel, p.S * p.Hkv, kSelThreads, (size_t)p.cached * 4, st, p);
    if (e == cudaSuccess) e = launch_pdl(rpa_evict_move_kernel, sms * 8, kMoveThreads, 0, st, p);
    return e;
}

}  // namespace rpa

using namespace rpa;

struct RpaEvict {
    RpaEvictCfg cfg;
    int device, sms;
    KernelSet ks;      // element types and scales of the attention of `cfg.cache`
    int weigh_bps;     // resident stats CTAs an SM
    int cached;
    void* ws;
    int* status;
    WeighParams w;     // workspace pointers and constants
    uint8_t* qbuf;     // q in the MMA operand type, where that is another
    int* list;
    int *seq_n, *seq_order;
};

namespace {

constexpr long long kMostLogits = 1ll << 28;  // floats: 1 GiB
constexpr int kMostPieces = 64;

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
    if (c->cache.kv_layout != RPA_KV_SPLIT) return RPA_ERR_UNSUPPORTED;
    // 32-bit row numbers, and grids of a CTA for each sequence and kv head
    if (c->cache.num_q_tokens * (c->cache.num_q_heads / c->cache.num_kv_heads) >= (int64_t)1 << 31 ||
        c->cache.max_num_seqs * c->cache.num_kv_heads >= (int64_t)1 << 31)
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
    if (weigh_prepare(h->ks.D, h->ks.kt, &h->weigh_bps) != cudaSuccess || h->weigh_bps < 1 ||
        compact_prepare((int)max_keys, &h->cached) != cudaSuccess) {
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
    double most = (double)small_rows * (double)Hkv * (double)max_keys;
    if (most > (double)kMostLogits) most = (double)kMostLogits;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t o_status = take(4), o_ctrl = take(16), o_stat0 = take((S + 1) * 4), o_item0 = take((S + 1) * 4),
                 o_block0 = take((S + 1) * 4), o_logit0 = take(S * 8), o_done = take(blocks * 4),
                 o_part = take((size_t)blocks * pieces * kWeighRows * 8), o_stat = take((size_t)blocks * kWeighRows * 8),
                 o_logits = take((size_t)most * 4), o_n = take(S * 4), o_order = take(S * 4),
                 o_list = take((size_t)S * Hkv * cfg->budget * 4),
                 o_q = take(h->ks.q_conv ? (size_t)c.num_q_tokens * c.num_q_heads * c.head_dim * 2 : 0);
    if (cudaMalloc(&h->ws, off) != cudaSuccess) {
        cudaGetLastError();
        delete h;
        return RPA_ERR_CUDA;
    }
    if (cudaMemset(h->ws, 0, 256) != cudaSuccess) {
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
    w.target = 4 * h->sms * h->weigh_bps;
    w.max_logits = (long long)most;
    w.status = h->status;
    w.ctrl = reinterpret_cast<int*>(b + o_ctrl);
    w.stat0 = reinterpret_cast<int*>(b + o_stat0);
    w.item0 = reinterpret_cast<int*>(b + o_item0);
    w.block0 = reinterpret_cast<int*>(b + o_block0);
    w.logit0 = reinterpret_cast<long long*>(b + o_logit0);
    w.done = reinterpret_cast<int*>(b + o_done);
    w.part = reinterpret_cast<float2*>(b + o_part);
    w.stat = reinterpret_cast<float2*>(b + o_stat);
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
        !aligned(cu_q_lens, 4) || !aligned(scores, 4))
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
    if (launch_weigh(p, h->ks.kt, h->sms * h->weigh_bps, st) != cudaSuccess) {
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
    if (!aligned(kv_pages, 16) || !aligned(scores, 4) || !aligned(kv_lens, 4) || !aligned(page_indices, 4) ||
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
    p.row_bytes = (int)(2 * c.head_dim * (kt_8bit(h->ks.kt) ? 1 : 2));
    p.budget = (int)h->cfg.budget;
    p.protect = (int)h->cfg.protect;
    p.recent = (int)h->cfg.recent;
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
