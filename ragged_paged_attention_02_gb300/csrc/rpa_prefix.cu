// rpa_prefix.cu -- attention of a batch whose sequences share their first keys (rpa_prefix_*).
//
// Softmax attention over keys A then B is the merge of the two partial results: with a part's maximum
// m_i, sum l_i and unnormalised O_i,  o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  So a group's shared
// keys can be attended by all of its query rows at once.  Decode on its own reads 2 D elements of every
// key for G rows; here B sequences of a group make B G rows of one kv head, dense tiles for the tensor
// cores, and the shared keys are read once a tile instead of once a sequence.
//
// The attention kernels are rpa_forward's, over another plan.  Every group becomes a virtual sequence:
// its query tokens are neighbours in q, its keys are the prefix, all visible to all of its tokens.  Every
// sequence stays one too, with the keys behind the prefix.  A virtual sequence with few rows (q_len * G of
// a decode tile) becomes pieces of the decode kernel, one with more becomes tiles of the prefill kernel, a
// prefix's tiles split over the keys as well.  Every item writes a partial; one merge takes each row's
// partials from both sources.
//
// As in rpa_forward the probabilities are rounded to the type of V's products (bf16 for bf16 K/V, else f16) before they meet
// V, and a q of another type than the products' is rounded to it; sums, maxima and partials are 32-bit.  With bf16 K/V and
// o a result is off by 2.2e-3 (root mean square, relative), of which 1.66e-3 are o's own rounding; with 8-bit K/V by 1.67e-3.
//
// How many pieces a prefix is cut into: tiles x kv heads are few (a batch of 64 and 8 heads has 8), so
// pieces fill the SMs; but each costs a pipeline ramp and 256 partial rows of D floats, written and read
// back.  The planner takes the number of pieces that makes  waves x (keys of a piece + kPieceCost)  least; where
// the sequences' pieces are items of the same kernel (8-bit pages), the larger of the longest item and the list's
// work a CTA: there fewer pieces, whose CTAs' gaps the others fill, take 65 us where a whole wave takes 69 (fp8).
//
// 61 sequences of 32 heads behind 8 k shared keys (bf16, D 128, 8 kv heads; 121 MB, 8.3 GFLOP): 49 us, of which plan
// 7, attention 34 and merge 7, 2.5 TB/s; 256 behind 16 k (593 MB, 71 GFLOP): 151 us, 3.9 TB/s and 470 TFLOP/s; 48 of
// three groups over fp8 pages (D 256; 99 MB): 65 us.  A sequence at a time the prefixes would be 2.0, 17 and
// 0.7 GB.  Bound by latencies: four dependent kernels, and in the attention kernels a few items an SM, each with its
// ramp (3.8 us a decode piece of 8-bit pages, where a tile of 64 keys takes 1.2).
#include <string.h>

#include <new>

#include "rpa_block.cuh"

namespace rpa {

namespace {

// FLOP/ns of one SM on a prefix's tiles beside the decode kernel: above rpa_forward's 6500 of prompt chunks, whose
// diagonal tiles are masked.  (256 x 16 k: 151 us a call from 8100 to 9300, 163 at 6500, 171 at 10800.)
constexpr int kPrefixSmGflops = 8700;
constexpr int kPieceAlign = 128;   // keys: the prefill kernels' tiles
constexpr int kPieceCost = 512;    // what a piece costs beside its keys, in keys (256: 167 us, 512 and 1024: 163, for 256 x 16 k)
constexpr int kUnitCost = 200;     // the same of a decode piece on the prefill kernel (3.8 us, where 64 keys take 1.2)
static_assert(kPlanThreads >= 160, "a candidate a thread");
constexpr int kMaxPieces = 160;    // most pieces of a prefix: one an SM where a single head and tile have all of them

struct PrefixPlan {
    const int *cu, *kv_lens, *cu_groups, *prefix_lens;
    int S, NG, T, Hkv, G, P, ps;
    int dec_rows, pf_tokens, pf_slots;  // rows of a decode tile; tokens and partial slots (of 16 rows) of a prefill tile
    int concurrent, n_sms, dec_bps, pf_bps, pf_mma_rows, dec_on_pf, D, kv_elt, dec_waves;
    int epoch;
    int max_dec_units, max_pf_units, max_part, item_room;
    int* ctrl;
    // per virtual sequence: groups 0 .. NG - 1, an empty one, sequences NG + 1 ..
    int *vcu, *vkv, *vrow;      // what the attention kernels read: first token, keys, row of the page table
    int4* vrec;                 // what the merge reads: first token, first partial slot, pieces (< 0: of prefill tiles)
    int2* token;                // [T]
    int* scratch;               // [kArrays, virtual sequences], used where they overflow shared memory
    Unit *dec_units, *pf_units;
};

constexpr int kArrays = 7;
constexpr int kVirtualSmem = 1536;  // virtual sequences whose records fit in shared memory (42 KB)

// The records of the virtual sequences: keys [begin, end) for ql tokens; class 0 no work, 1 decode pieces, 2 prefill
// tiles; units of each kind (decode pieces: of sequences of more than half a piece, then of the others) up to and with this one
struct Records {
    int *q0, *ql, *begin, *end, *long_end, *short_end, *pf_end;
    __device__ __forceinline__ int cls(const PrefixPlan& p, int v) const {
        return ql[v] == 0 || end[v] <= begin[v] ? 0 : (long long)ql[v] * p.G <= p.dec_rows ? 1 : 2;
    }
};

// Sums of a and b and the largest m over the block, and whether any thread found a fault: one round of barriers
__device__ __forceinline__ bool block_totals(unsigned long long& a, unsigned long long& b, int& m, bool bad, unsigned long long* s_red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) {
        s_red[warp] = a;
        s_red[32 + warp] = b;
        s_red[64 + warp] = (unsigned long long)m;
    }
    if (__syncthreads_or(bad)) return true;
    a = lane < nwarps ? s_red[lane] : 0ull;
    b = lane < nwarps ? s_red[32 + lane] : 0ull;
    m = __reduce_max_sync(0xffffffffu, lane < nwarps ? (int)s_red[64 + lane] : 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return false;
}

// The warp's least cost and its candidate, the lowest of equal costs
__device__ __forceinline__ void warp_least(float& cost, int& candidate) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float c = __shfl_xor_sync(0xffffffffu, cost, o);
        const int x = __shfl_xor_sync(0xffffffffu, candidate, o);
        if (c < cost || (c == cost && x < candidate)) {
            cost = c;
            candidate = x;
        }
    }
}

__global__ void __launch_bounds__(kPlanThreads, 1) rpa_prefix_plan_kernel(const PrefixPlan p) {
    __shared__ int s_rec[kArrays * kVirtualSmem];
    __shared__ int s_scan[33 * 4];
    __shared__ unsigned long long s_red[96];
    const int tid = threadIdx.x, lane = tid & 31, S = p.S, NG = p.NG, V = S > 0 ? NG + 1 + S : 0;
    int* ctrl = p.ctrl;
    const int Tq = p.pf_tokens;
    Records R;
    {
        int* base = V <= kVirtualSmem ? s_rec : p.scratch;
        const int n = V <= kVirtualSmem ? kVirtualSmem : V;
        int** to[kArrays] = {&R.q0, &R.ql, &R.begin, &R.end, &R.long_end, &R.short_end, &R.pf_end};
#pragma unroll
        for (int i = 0; i < kArrays; ++i) *to[i] = base + (size_t)i * n;
    }
    pdl_trigger();
    pdl_wait();
    auto give_up = [&](int code) {  // no items; the merge writes zeros
        if (tid == 0) {
            for (int w = 1; w < kCtrlWords; ++w) ctrl[w] = 0;
            ctrl[kNumComb] = -1;
            set_status(ctrl, code);
            publish_epoch(ctrl, p.epoch);
        }
    };
    // ---- 1. records, checks, and the work of the two kernels: key x kv head pairs of decode pieces, tile x key x kv
    // head of prefill tiles.  A group's bounds are checked by its own thread; a sequence's lookup of its group stays
    // in range whatever they hold.
    bool bad = tid == 0 && (NG > 0 ? p.cu_groups[0] != 0 || p.cu_groups[NG] != S : S != 0);
    unsigned long long dec_keys = 0, pf_keys = 0;
    int longest = 0;
    for (int v = tid; v < max(V, NG); v += kPlanThreads) {
        int q0 = 0, ql = 0, begin = 0, end = 0, row = 0;
        if (v < NG) {
            const int a = p.cu_groups[v], b = p.cu_groups[v + 1];
            end = p.prefix_lens[v];
            if (a < 0 || b < a || b > S || end < 0 || end > p.P * p.ps) {
                bad = true;
                end = 0;
            } else {
                row = a;
                q0 = p.cu[a];
                ql = p.cu[b] - q0;
            }
        } else if (v == NG) {
            q0 = p.cu[S];  // the last group's end: the pair (v, v + 1) of every other virtual sequence is its tokens
        } else {
            row = v - NG - 1;
            q0 = p.cu[row];
            ql = p.cu[row + 1] - q0;
            end = p.kv_lens[row];
            if (NG > 0) begin = p.prefix_lens[upper_seq(p.cu_groups + 1, NG, row)];
            if (q0 < 0 || ql < 0 || end < 0 || end > p.P * p.ps || ql > end || q0 + (long long)ql > p.T || (ql > 0 && begin > end - ql)) {
                bad = true;
                ql = 0;
            }
        }
        if (v >= V) continue;
        R.q0[v] = q0;
        R.ql[v] = ql;
        R.begin[v] = begin;
        R.end[v] = end;
        p.vrow[v] = row;
        const int cls = R.cls(p, v), keys = end - begin;
        if (cls == 1) dec_keys += (unsigned long long)keys * p.Hkv;
        if (cls == 2) {
            pf_keys += (unsigned long long)((ql + Tq - 1) / Tq) * (unsigned long long)keys * p.Hkv;
            if (v < NG) longest = max(longest, end);
        }
    }
    if (tid == 0 && V > 0) p.vcu[V] = p.cu[S];
    if (block_totals(dec_keys, pf_keys, longest, bad, s_red)) {
        give_up(RPA_ERR_BAD_LENGTHS);
        return;
    }
    // ---- 2. SMs of each kernel when both run at once: x SMs of prefill take F / (x a), the others B / ((n - x) d);
    // they end together where F d (n - x) = B a x
    int pf_ctas = p.n_sms * p.pf_bps, dec_ctas = p.n_sms * p.dec_bps;
    if (p.concurrent && dec_keys && pf_keys) {
        const float B = (float)dec_keys * (float)(2 * p.D * p.kv_elt), F = (float)pf_keys * (float)p.pf_mma_rows * (float)(4 * p.D);
        const float fd = F * (float)kDecSmGBs, ba = B * (float)kPrefixSmGflops;
        int x = (int)((float)p.n_sms * fd / (fd + ba) + 0.5f);
        x = min(max(x, 1), p.n_sms - 1);
        pf_ctas = x * p.pf_bps;
        dec_ctas = (p.n_sms - x) * p.dec_bps;
    }
    // ---- 3. keys of a decode piece, and of a piece of a prefix's tiles
    const int on = p.dec_on_pf ? pf_ctas : dec_ctas;
    const unsigned long long want = dec_keys / (unsigned long long)max(1, p.dec_waves * on) + 1;
    const int chunk = (int)min(max((want + kChunkAlign - 1) / kChunkAlign * kChunkAlign, (unsigned long long)kMinChunk), 1ull << 30);
    int pf_chunk = kPieceAlign;
    if (longest > 0) {
        // pieces of the longest prefix: a candidate a thread, the warps' bests by cost and then by number
        float cost = INFINITY;
        if (tid < kMaxPieces) {
            const int c = ((longest + tid) / (tid + 1) + kPieceAlign - 1) / kPieceAlign * kPieceAlign;
            long long items = 0, fewest = 0;
            for (int g = 0; g < NG; ++g) {
                if (R.cls(p, g) != 2) continue;
                const int tiles = (R.ql[g] + Tq - 1) / Tq * p.Hkv;
                items += (long long)tiles * ((R.end[g] + c - 1) / c);
                fewest += tiles;
            }
            // (whole waves of whole keys: exact in a float up to 2^24, and far from it where a choice is close)
            if (tid == 0 || items <= fewest + p.item_room) {
                // the decode pieces' keys fill the CTAs that have no prefix tile, where they are items of the same kernel
                const float others = (float)(pf_keys + dec_keys) + (float)S * (float)(p.Hkv * kUnitCost);
                cost = p.dec_on_pf ? fmaxf((float)(c + kPieceCost), ((float)items * kPieceCost + others) / (float)pf_ctas)
                                   : ceilf((float)items / (float)pf_ctas) * (float)(c + kPieceCost);
            }
        }
        float* costs = reinterpret_cast<float*>(s_red);
        int* who = reinterpret_cast<int*>(s_red + 32);
        int best = tid;
        warp_least(cost, best);
        __syncthreads();  // block_totals' reads
        if (lane == 0) {
            costs[tid >> 5] = cost;
            who[tid >> 5] = best;
        }
        __syncthreads();
        cost = lane < kPlanThreads / 32 ? costs[lane] : INFINITY;
        best = lane < kPlanThreads / 32 ? who[lane] : kMaxPieces;
        warp_least(cost, best);
        pf_chunk = ((longest + best) / (best + 1) + kPieceAlign - 1) / kPieceAlign * kPieceAlign;
    }
    // ---- 4. units and partial slots of each virtual sequence
    int n_long = 0, n_short = 0, n_pf = 0, n_part = 0;
    for (int base = 0; base < V; base += kPlanThreads) {
        const int v = base + tid;
        int add[4] = {0, 0, 0, 0}, off[4], tot[4], cls = 0, pieces = 0;
        if (v < V) {
            cls = R.cls(p, v);
            if (cls == 1) {
                pieces = (R.end[v] - R.begin[v] + chunk - 1) / chunk;
                add[R.end[v] - R.begin[v] > chunk / 2 ? 0 : 3] = pieces;
                add[2] = pieces * p.Hkv;
            } else if (cls == 2) {
                pieces = v < NG ? (R.end[v] + pf_chunk - 1) / pf_chunk : 1;
                add[1] = (R.ql[v] + Tq - 1) / Tq * pieces;
                add[2] = add[1] * p.Hkv * p.pf_slots;
            }
        }
        block_scan<4>(add, off, tot, s_scan);
        if (v < V) {
            p.vcu[v] = R.q0[v];
            // positions behind the prefix: a group's keys are visible to all of its tokens
            p.vkv[v] = v < NG ? R.end[v] + R.ql[v] : R.end[v];
            p.vrec[v] = make_int4(R.q0[v], n_part + off[2], cls == 2 ? -pieces : pieces, 0);
            R.long_end[v] = n_long + off[0] + add[0];
            R.short_end[v] = n_short + off[3] + add[3];
            R.pf_end[v] = n_pf + off[1] + add[1];
        }
        n_long += tot[0];
        n_short += tot[3];
        n_pf += tot[1];
        n_part += tot[2];
    }
    const int n_dec = n_long + n_short, n_list = p.dec_on_pf ? n_pf + n_dec : n_pf;
    if (n_dec > p.max_dec_units || n_list > p.max_pf_units || n_part > p.max_part) {
        give_up(RPA_ERR_INVALID_ARG);  // cannot happen with the create-time sizing; refuse rather than overflow
        return;
    }
    __syncthreads();
    // ---- 5. the unit lists: prefix tiles first, a piece's tiles together (they share its keys); then the decode pieces,
    // the longer ones first, so that short ones even out the end (61 x 8 k: 49.8 -> 48.9 us; the others as before)
    for (int u = tid; u < n_dec + n_pf; u += kPlanThreads) {
        const bool dec = u >= n_pf;
        const int x = dec ? u - n_pf : u, of = dec && x >= n_long ? x - n_long : x;  // of: its number in its list
        const int* ends = !dec ? R.pf_end : x < n_long ? R.long_end : R.short_end;
        const int v = upper_seq(ends, V, of);
        const int4 rec = p.vrec[v];
        const int first = v > 0 ? ends[v - 1] : 0, k = of - first;
        int4 a, b;
        if (dec) {
            const int kb = R.begin[v] + k * chunk;
            a = make_int4(v, 0, R.ql[v], kb);
            b = make_int4(min(R.end[v], kb + chunk), rec.y, k, rec.z);
        } else {
            const int ql = R.ql[v], end = R.end[v], pieces = -rec.z;
            const int tiles = (ql + Tq - 1) / Tq, tile = k % tiles, piece = k / tiles;
            const int t0 = tile * Tq, nt = min(Tq, ql - t0);
            const int kb = v < NG ? piece * pf_chunk : R.begin[v];
            const int ke = v < NG ? min(end, kb + pf_chunk) : min(end, end - ql + t0 + nt);
            a = make_int4(v, t0, nt, kb);
            b = make_int4(ke, rec.y + tile * p.Hkv * pieces * p.pf_slots, piece * p.pf_slots, pieces * p.pf_slots);
        }
        Unit* dst = dec && !p.dec_on_pf ? p.dec_units + x : p.pf_units + u;
        reinterpret_cast<int4*>(dst)[0] = a;
        reinterpret_cast<int4*>(dst)[1] = b;
    }
    // ---- 6. each token's virtual sequences
    const int t_lo = S > 0 ? R.q0[NG + 1] : 0, t_hi = S > 0 ? R.q0[NG] : 0;
    for (int t = tid; t < p.T; t += kPlanThreads) {
        int2 who = make_int2(-1, -1);
        if (t >= t_lo && t < t_hi) {
            const int s = upper_seq(R.q0 + NG + 2, S, t);  // the first whose successor starts behind t
            who = make_int2(upper_seq(p.cu_groups + 1, NG, s), NG + 1 + s);
        }
        p.token[t] = who;
    }
    __syncthreads();  // (publish_epoch's fence covers what the barrier has gathered)
    if (tid == 0) {
        ctrl[kNumDecItems] = p.dec_on_pf ? 0 : n_dec * p.Hkv;
        ctrl[kNumPfItems] = n_list * p.Hkv;
        ctrl[kNumComb] = 0;
        ctrl[kDecChunk] = chunk;
        ctrl[kDecCounter] = 0;
        ctrl[kPfCounter] = 0;
        ctrl[kNumPart] = n_part;
        ctrl[kNumUnits] = n_dec + n_pf;
        ctrl[kPfCtas] = pf_ctas;
        ctrl[kDecCtas] = dec_ctas;
        publish_epoch(ctrl, p.epoch);
    }
}

// ---------------------------------------------------------------- merge
struct PrefixMerge {
    uint8_t* o;
    const int2* token;  // [T] virtual sequences of a token's group and of its sequence (y -1: of none)
    const int4* vrec;   // [virtual sequences] first token, first partial slot, pieces (< 0: of prefill tiles)
    const int* ctrl;
    int T, Hq, Hkv, G, D;
    int pf_tokens, pf_slots;
    int per_token;  // CTAs of a token
    float v_scale;
    const float* sinks;
    int odt;
    const float *part_o, *part_ml;
};

constexpr int kMergeThreads = 256;

// A row's partials of one virtual sequence: row `row` of slots slot, slot + stride, ...
struct Source {
    int slot, stride, n, row;
};
__device__ __forceinline__ Source source(const PrefixMerge& p, const int4& v, int t, int h, int g) {
    Source r;
    const int pieces = v.z, tl = t - v.x;
    r.n = pieces < 0 ? -pieces : pieces;
    if (pieces >= 0) {
        r.slot = v.y + h * pieces;
        r.stride = 1;
        r.row = tl * p.G + g;
    } else {
        // a prefill tile: one or (16 slots) two halves of 128 rows
        const int tile = tl / p.pf_tokens, tt = tl - tile * p.pf_tokens;
        const int half_tokens = p.pf_slots == 16 ? p.pf_tokens / 2 : p.pf_tokens;
        r.stride = p.pf_slots;
        r.slot = v.y + (tile * p.Hkv + h) * r.n * p.pf_slots;
        r.row = tt / half_tokens * kTcRows + tt % half_tokens * p.G + g;
    }
    return r;
}

__global__ void __launch_bounds__(kMergeThreads, 4) rpa_prefix_merge_kernel(const PrefixMerge p) {
    constexpr int kBatch = 8;  // partial O loads a lane has in flight
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, t = blockIdx.x / p.per_token;
    const int task = (blockIdx.x - t * p.per_token) * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int quads = p.D / 4, chunks = (quads + 31) / 32;  // 128-column chunks of a row
    if (task >= p.Hq * chunks) return;
    const int qh = task / chunks, c4 = (task - qh * chunks) * 32 + lane;
    const bool act = c4 < quads;
    const int2 who = p.token[t];  // virtual sequences of the token's group and of its sequence
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float inv = 0.f;
    if (who.y >= 0 && p.ctrl[kNumComb] >= 0) {
        const int h = qh / p.G, g = qh - h * p.G;
        const int4 va = p.vrec[who.x], vb = p.vrec[who.y];
        const Source a = source(p, va, t, h, g), b = source(p, vb, t, h, g);
        const int n = a.n + b.n;
        // this lane's four columns in a slot's rows: row-major, or the prefill kernel's blocks of eight columns
        const bool a_blocked = va.z < 0 && p.pf_slots == 16, b_blocked = vb.z < 0 && p.pf_slots == 16;
        const int blocked = (c4 / 2) * (2 * kTcRows * 8) + (c4 & 1) * 4;
        float M = -INFINITY, L = 0.f;
        for (int k0 = 0; k0 < n; k0 += 32) {
            // lane k: partial k0 + k
            const int k = k0 + lane;
            const bool in_a = k < a.n;
            const int slot = in_a ? a.slot + k * a.stride : b.slot + (k - a.n) * b.stride;
            const float2 ml = k < n ? *reinterpret_cast<const float2*>(p.part_ml + ((size_t)slot * kDecRows + (in_a ? a.row : b.row)) * 2)
                                    : make_float2(-INFINITY, 0.f);
            const int most = min(32, n - k0);
            float4 x[kBatch];
            auto fetch = [&](int j0) {
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const int kk = k0 + j0 + j;
                    if (act && j0 + j < most) {
                        const bool ina = kk < a.n;
                        const int sl = ina ? a.slot + kk * a.stride : b.slot + (kk - a.n) * b.stride, row = ina ? a.row : b.row;
                        const float* o = p.part_o + (size_t)sl * kDecRows * p.D;
                        o += (ina ? a_blocked : b_blocked) ? blocked + row * 8 : row * p.D + c4 * 4;
                        x[j] = __ldcs(reinterpret_cast<const float4*>(o));
                    }
                }
            };
            fetch(0);  // beside the maxima and sums
            float m = ml.x;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float Mn = fmaxf(M, m), keep = M == -INFINITY ? 0.f : ex2(M - Mn);
            // a part whose keys are all hidden has no maximum and joins with weight 0
            const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - Mn);
            float l = w * ml.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            L = L * keep + l;
            M = Mn;
            acc.x *= keep; acc.y *= keep; acc.z *= keep; acc.w *= keep;
            for (int j0 = 0; j0 < most; j0 += kBatch) {
                if (j0 > 0) fetch(j0);
#pragma unroll
                for (int j = 0; j < kBatch; ++j) {
                    const float wj = __shfl_sync(0xffffffffu, w, (j0 + j) & 31);
                    if (act && j0 + j < most) {
                        acc.x += wj * x[j].x;
                        acc.y += wj * x[j].y;
                        acc.z += wj * x[j].z;
                        acc.w += wj * x[j].w;
                    }
                }
            }
        }
        L = add_sink(L, p.sinks, qh, M);
        inv = L > 0.f ? p.v_scale / L : 0.f;
        if (M == -INFINITY) acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    if (act)
        store_o4(p.o, ((size_t)t * p.Hq + qh) * p.D + 4 * c4, acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv, p.odt);
}

}  // namespace
}  // namespace rpa

using namespace rpa;

struct RpaPrefix {
    RpaCfg cfg;
    int64_t max_groups;
    int device;
    KernelSet ks;
    void* ws;
    Workspace w;
    int pf_slots, item_room, max_dec_units, max_pf_units, max_part;
    int *vcu, *vkv, *vrow, *scratch;
    int4* vrec;
    int2* token;
    cudaStream_t side;
    cudaEvent_t ev_plan, ev_dec;
    int epoch;
};

namespace {

void prefix_free(RpaPrefix* h) {
    if (h->ev_dec) cudaEventDestroy(h->ev_dec);
    if (h->ev_plan) cudaEventDestroy(h->ev_plan);
    if (h->side) cudaStreamDestroy(h->side);
    if (h->ws) cudaFree(h->ws);
    delete h;
}

bool prefix_allocate(RpaPrefix* h) {
    const RpaCfg& c = h->cfg;
    KernelSet& ks = h->ks;
    int sms = 0;
    if (cudaGetDevice(&h->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, h->device) != cudaSuccess)
        return false;
    kernels_choose(c, sms, &ks);
    if (kernels_prepare(c, &ks) != cudaSuccess) return false;
    // worst cases.  Decode: a piece of each virtual sequence, and dec_waves pieces a CTA.  Prefill tiles: of T tokens
    // and one part-empty tile a virtual sequence of that class (more than dec_rows rows), item_room pieces more
    const int64_t S = c.max_num_seqs, T = c.num_q_tokens, Hkv = ks.Hp, NG = h->max_groups, Tq = ks.pf_tokens;
    h->pf_slots = ks.tc ? 16 : 8;
    h->item_room = 4 * sms * ks.pf_bps;
    const int64_t big = T * ks.G / (ks.dec_rows + 1);  // sequences, or groups, of the prefill class
    const int64_t group_tiles = T / Tq + (NG < big ? NG : big) + 1, seq_tiles = T / Tq + (S < big ? S : big) + 1;
    const int64_t dec_units = S + NG + (kDecWaves * (int64_t)sms * ks.dec_bps + Hkv - 1) / Hkv + 1;
    const int64_t pf_units = group_tiles + seq_tiles + h->item_room / Hkv + 1;
    const int64_t part = dec_units * Hkv + pf_units * Hkv * h->pf_slots;  // (pf_units holds the item_room pieces)
    if (part >= ((int64_t)1 << 31) / kDecRows) return false;
    h->max_dec_units = (int)dec_units;
    h->max_pf_units = (int)(ks.tc8 ? pf_units + dec_units : pf_units);
    h->max_part = (int)part;
    const size_t V = (size_t)(NG + S + 2);
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = (off + bytes + 255) & ~(size_t)255;
        return at;
    };
    const size_t o_ctrl = take(kCtrlWords * sizeof(int)), o_v = take(3 * V * sizeof(int)), o_rec = take(V * sizeof(int4)),
                 o_scratch = take(V > kVirtualSmem ? kArrays * V * sizeof(int) : 0), o_token = take((size_t)T * sizeof(int2)),
                 o_dec = take((size_t)h->max_dec_units * sizeof(Unit)), o_pf = take((size_t)h->max_pf_units * sizeof(Unit)),
                 o_po = take((size_t)part * kDecRows * ks.D * sizeof(float)), o_ml = take((size_t)part * kDecRows * 2 * sizeof(float)),
                 o_q = take(ks.q_conv ? (size_t)T * c.num_q_heads * ks.D * 2 : 0);
    if (cudaMalloc(&h->ws, off) != cudaSuccess) return false;
    if (!set_now(cudaMemset(h->ws, 0, kCtrlWords * sizeof(int)))) return false;
    uint8_t* b = static_cast<uint8_t*>(h->ws);
    h->w.ctrl = reinterpret_cast<int*>(b + o_ctrl);
    h->w.dec_units = reinterpret_cast<Unit*>(b + o_dec);
    h->w.pf_units = reinterpret_cast<Unit*>(b + o_pf);
    h->w.part_o = reinterpret_cast<float*>(b + o_po);
    h->w.part_ml = reinterpret_cast<float*>(b + o_ml);
    h->w.qbuf = ks.q_conv ? b + o_q : nullptr;
    int* v = reinterpret_cast<int*>(b + o_v);
    h->vcu = v;
    h->vkv = v + V;
    h->vrow = v + 2 * V;
    h->vrec = reinterpret_cast<int4*>(b + o_rec);
    h->scratch = reinterpret_cast<int*>(b + o_scratch);
    h->token = reinterpret_cast<int2*>(b + o_token);
    return !ks.tc || (cudaStreamCreateWithFlags(&h->side, cudaStreamNonBlocking) == cudaSuccess &&
                      cudaEventCreateWithFlags(&h->ev_plan, cudaEventDisableTiming) == cudaSuccess &&
                      cudaEventCreateWithFlags(&h->ev_dec, cudaEventDisableTiming) == cudaSuccess);
}

}  // namespace

extern "C" {

int rpa_prefix_validate_cfg(const RpaCfg* cfg, int64_t max_groups) {
    const int v = rpa_validate_cfg(cfg);
    if (v != RPA_OK) return v;
    if (max_groups < 1 || max_groups > cfg->max_num_seqs) return RPA_ERR_INVALID_ARG;
    if (cfg->kv_layout != RPA_KV_SPLIT || !cfg->is_causal || cfg->has_sliding_window) return RPA_ERR_UNSUPPORTED;
    // keys and a piece's, positions of a group's tokens behind its prefix, and rows of the virtual batch, in 32 bits
    if (cfg->pages_per_seq * cfg->page_size > (int64_t)1 << 30 || cfg->num_q_tokens >= (int64_t)1 << 30 ||
        cfg->num_q_tokens * cfg->num_q_heads >= (int64_t)1 << 31)
        return RPA_ERR_UNSUPPORTED;
    return RPA_OK;
}

int rpa_prefix_create(const RpaCfg* cfg, int64_t max_groups, RpaPrefix** out) {
    if (!out) return RPA_ERR_INVALID_ARG;
    *out = nullptr;
    const int v = rpa_prefix_validate_cfg(cfg, max_groups);
    if (v != RPA_OK) return v;
    RpaPrefix* h = new (std::nothrow) RpaPrefix;
    if (!h) return RPA_ERR_CUDA;
    memset(h, 0, sizeof *h);
    h->cfg = *cfg;
    h->max_groups = max_groups;
    if (!prefix_allocate(h)) {
        cudaGetLastError();
        prefix_free(h);
        return RPA_ERR_CUDA;
    }
    *out = h;
    return RPA_OK;
}

int rpa_prefix_forward(RpaPrefix* h, const void* q, const void* kv_pages, const int32_t* kv_lens,
                       const int32_t* page_indices, const int32_t* cu_q_lens, int32_t num_seqs, const int32_t* cu_groups,
                       const int32_t* prefix_lens, int32_t num_groups, void* o, void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    const RpaCfg& c = h->cfg;
    const KernelSet& ks = h->ks;
    if (num_seqs < 0 || num_seqs > c.max_num_seqs) return RPA_ERR_INVALID_ARG;
    if (num_groups < 0 || num_groups > h->max_groups || (num_groups == 0 && num_seqs > 0)) return RPA_ERR_INVALID_ARG;
    if (!kv_pages || !kv_lens || !page_indices || !cu_q_lens) return RPA_ERR_INVALID_ARG;
    if (num_groups > 0 && (!cu_groups || !prefix_lens)) return RPA_ERR_INVALID_ARG;
    if (c.num_q_tokens > 0 && (!q || !o)) return RPA_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(o, 16) || !aligned(kv_pages, 16) || !aligned(kv_lens, 4) || !aligned(page_indices, 4) ||
        !aligned(cu_q_lens, 4) || !aligned(cu_groups, 4) || !aligned(prefix_lens, 4))
        return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    if (!g.ok) return RPA_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const void* qk = q;
    if (c.num_q_tokens > 0 && ks.q_conv) {
        const size_t n = (size_t)c.num_q_tokens * c.num_q_heads * ks.D;
        if (launch_q_convert(q, c.q_dtype, h->w.qbuf, ks.q_conv_f16, n, Launch{ks.sms * 4, st}) != cudaSuccess) {
            cudaGetLastError();
            return RPA_ERR_CUDA;
        }
        qk = h->w.qbuf;
    }
    EnqueueOpts eo;
    memset(&eo, 0, sizeof eo);
    eo.st = st;
    eo.conc = ks.tc;
    eo.side = h->side;
    eo.ev_plan = h->ev_plan;
    eo.ev_dec = h->ev_dec;
    eo.timeout_ns = 1000000000ull;
    eo.epoch = h->epoch = (h->epoch + 1) & 0x7FFFFFFF;
    PrefixPlan p;
    p.cu = cu_q_lens;
    p.kv_lens = kv_lens;
    p.cu_groups = cu_groups;
    p.prefix_lens = prefix_lens;
    p.S = num_seqs;
    p.NG = num_groups;
    p.T = (int)c.num_q_tokens;
    p.Hkv = ks.Hp;
    p.G = ks.G;
    p.P = (int)c.pages_per_seq;
    p.ps = (int)c.page_size;
    p.dec_rows = ks.dec_rows;
    p.pf_tokens = ks.pf_tokens;
    p.pf_slots = h->pf_slots;
    p.concurrent = eo.conc;
    p.n_sms = ks.sms;
    p.dec_bps = ks.dec_bps;
    p.pf_bps = ks.pf_bps;
    p.pf_mma_rows = ks.tc ? 2 * kTcRows : kTcRows;
    p.dec_on_pf = ks.tc8;
    p.D = ks.D;
    p.kv_elt = kt_8bit(ks.kt) ? 1 : 2;
    p.dec_waves = ks.tc8 ? kDecWavesTc8 : kDecWaves;
    p.epoch = eo.epoch;
    p.max_dec_units = h->max_dec_units;
    p.max_pf_units = h->max_pf_units;
    p.max_part = h->max_part;
    p.item_room = h->item_room;
    p.ctrl = h->w.ctrl;
    p.vcu = h->vcu;
    p.vkv = h->vkv;
    p.vrow = h->vrow;
    p.vrec = h->vrec;
    p.token = h->token;
    p.scratch = h->scratch;
    p.dec_units = h->w.dec_units;
    p.pf_units = h->w.pf_units;
    if (launch_pdl(rpa_prefix_plan_kernel, 1, kPlanThreads, 0, st, p) != cudaSuccess) {
        cudaGetLastError();
        return RPA_ERR_CUDA;
    }
    AttnParams ap = attn_params(c, ks, h->w, qk, kv_pages, h->vkv, page_indices, h->vcu, o);
    ap.page_rows = h->vrow;
    MapCache maps = {};
    const int r = enqueue_attention(c, ks, h->w, &maps, ap, eo);
    if (r != RPA_OK) {
        cudaGetLastError();
        return r;
    }
    if (c.num_q_tokens == 0) return RPA_OK;
    PrefixMerge m;
    m.o = static_cast<uint8_t*>(o);
    m.token = h->token;
    m.vrec = h->vrec;
    m.ctrl = h->w.ctrl;
    m.T = (int)c.num_q_tokens;
    m.Hq = (int)c.num_q_heads;
    m.Hkv = ks.Hp;
    m.G = ks.G;
    m.D = ks.D;
    m.pf_tokens = ks.pf_tokens;
    m.pf_slots = h->pf_slots;
    m.per_token = (m.Hq * ((m.D + 127) / 128) + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
    m.v_scale = ks.v_scale;
    m.sinks = ap.sinks;
    m.odt = ks.odt;
    m.part_o = h->w.part_o;
    m.part_ml = h->w.part_ml;
    if (launch_pdl(rpa_prefix_merge_kernel, m.T * m.per_token, kMergeThreads, 0, st, m) != cudaSuccess) {
        cudaGetLastError();
        return RPA_ERR_CUDA;
    }
    return RPA_OK;
}

int rpa_prefix_get_status(RpaPrefix* h, void* stream) {
    if (!h) return RPA_ERR_INVALID_ARG;
    DeviceGuard g(h->device);
    return g.ok ? take_status(h->w.ctrl + kStatus, static_cast<cudaStream_t>(stream)) : RPA_ERR_CUDA;
}

void rpa_prefix_destroy(RpaPrefix* h) {
    if (!h) return;
    DeviceGuard g(h->device);
    prefix_free(h);
}

}  // extern "C"
