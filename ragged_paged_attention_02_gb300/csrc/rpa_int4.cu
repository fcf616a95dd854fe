// rpa_int4.cu -- attention over a cache of 4-bit codes.
//
// A channel of a key is  code * s + z  with a scale s and a zero z of its group of channels, so a logit and an output are
//   q . k  = sum over groups  s_g (q . code)_g + z_g (sum of q)_g
//   o      = sum over keys  p s code + p z
//          = sum over keys  P code  -  8 sum over keys P  +  sum over keys p (z + 8 s),     P = f16(p s)
// The matrix products run on the codes themselves, exact in f16; scales and zeros act on 32-bit sums of a group and on the
// probabilities.  P is the only rounded factor, and its rounding meets code - 8, at most half a group's range: with the codes
// 0 .. 15 alone it would be twice to three times as large.  Sums of P come out of one more product, with ones.
//
// Codes become f16 operands with a mask: bits 0 - 3 of a 16-bit word are the subnormal code * 2^-24, bits 4 - 7 code * 2^-20,
// and 8 bits further down the same again (5 instructions for 8 codes).  Codes of the two positions go to different accumulators
// (logits) or output rows (values), whose powers of two are applied at the end.  q is rounded to f16.
//
//  * direct kernel: tiles of 8 query rows (tokens x heads of a kv head).  Keys are on the M side of m16n8k16: S^T = K Q^T,
//    O^T += V^T P^T, so that one decoded operand serves all rows; matrix loads of 16-bit units give a thread four codes of a key
//    (K) or of two keys (V, transposed) just as the operands want them.  One producer warp copies whole blocks of a page and kv
//    head (or four pieces of one where its size is not that of a run) into a ring of stages, the other warps take 32 keys of
//    each.  Bound by instructions more than by bytes (a key and kv head costs 17 issue slots at D 128, of the 25 that its bytes'
//    time has), so as few warps as can feed the others issue copies.  (Warps that each copied for themselves took 25.)
//    128 decodes of 512 to 16 k keys (32 query and 8 kv heads, D 128, groups of 64, 1245 MB): 225 us of the call's 232, 5.5 TB/s.
//    16 decodes of a 4 k window (D 256, groups of 128, soft cap, 143 MB): 43 us of 51, 3.4 TB/s (64 of them 125 us, 4.5 TB/s): some
//    45 instructions a key and warp, which 12 warps of 168 registers issue in 39 % of the cycles; three to five consumer warps,
//    two or three CTAs an SM, and pieces of 4 to 13 stages all took 53 to 59 us where this took 54.  32 sequences of 1 to 5
//    tokens (D 64, 35 MB, some keys in two or three tiles): 24 us of 35, issue 54 %.  4 decodes: 17 us a call, 8 of them
//    dependent loads and the planner's latency before the first product.
//    Smaller groups cost more: a scale, a zero, a transposed P and its sum for each (16 decodes at D 256 as above: 52 us with groups of
//    128, 70 of 64, 109 of 32, which spill).
//  * long prompts would decode every key once for each tile.  Sequences with more tokens are unfolded instead, once a call, to
//    f16 rows in the workspace, over which the tensor-memory prefill kernels run.  Three prompts of 0.8 to 2 k tokens on top
//    of 4 to 16 k keys (32 and 8 heads, D 128): 529 us, 40 of them the rows (and q's rounding; 203 MB, 5.1 TB/s) and 468 the
//    attention (562 GFLOP, 1.2 PFLOP/s).
#include <cuda_fp16.h>
#include <string.h>

#include "rpa_evict.cuh"  // FastDiv
#include "rpa_internal.cuh"

namespace rpa {
namespace {

constexpr int R = kInt4Rows;
// The running maximum moves when a row's grows by more than 2^2: probabilities stay below 4, and P below 4 * 8736 (the
// greatest scale of float16 values), in f16's range
constexpr float kRescale = 2.f;

struct I4Params {
    AttnParams a;            // a.G: query heads of an item (the last block of a kv head may have fewer); a.Hkv: the cache's
    int heads, blocks;       // query heads of a kv head, and the items' heads they make
    int BR, brs;             // keys of a copied page run, log2
    uint32_t block;          // bytes of a page's block
    FastDiv page;            // by the page size
    int most_items;          // that the list has room for
    int stall;               // test hook (RPA_OPT_TEST_STALL_PRODUCER)
    unsigned long long timeout_ns;
};

// words of a stage's description: four in one load each
enum I4Meta : int { mKey0 = 0, mKvBegin, mKvEnd, mLeft, mPos, mNtok, mSwz, mFirst, mHead, mTok, mPart, mHeads, mSwz2, kMetaWords = 16 };

template <int D, int NG>
struct I4Geom {
    static constexpr int CW = int4_warps(D);          // consumer warps
    static constexpr int THREADS = (CW + 1) * 32;
    static constexpr int KS = 32 * CW;                // keys of a stage
    static constexpr int KB = D + 8 * NG;             // bytes of a key
    static constexpr int STAGE = KS * KB;
    static constexpr int QB = R * D * 2;              // Q of an item
    // D 256: Q's operands in shared memory, one copy for all warps (in registers they made the loop spill, 54 -> 52 us below)
    static constexpr bool QSH = D == 256;
    static constexpr int QF = QSH ? R * D * 2 : 0;
    static constexpr int LD = D + 4;                  // floats of a row of the merge area: rows of four lanes fall into different banks
    static constexpr int RED = CW * R * LD * 4;       // ... which lies in the item's last stage
    // resident CTAs that registers are allocated for, and stages: as many as fit beside them
    static constexpr int CTAS = 2;
    static constexpr int FIT = (227 * 1024 / CTAS - 3 * 1024 - QB - QF) / STAGE;
    static constexpr int NS = FIT > 4 ? 4 : FIT;
    static constexpr int SMEM = NS * STAGE + QB + QF;
    static_assert(NS >= 2 && RED <= STAGE, "a ring; the merge area");
};

__device__ __forceinline__ void bulk_copy(uint32_t dst, const uint8_t* src, uint32_t bytes, uint32_t bar, uint64_t pol) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;\n" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar), "l"(pol)
        : "memory");
}
// 8 x 8 matrix of 16-bit elements, transposed across the warp
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// Eight neighbouring 16-bit q values (global or shared) as f16 pairs, rounded to nearest even
__device__ __forceinline__ uint4 load_q8(const uint8_t* q, size_t e, int bf16) {
    uint4 w = *reinterpret_cast<const uint4*>(q + e * 2);
    if (bf16) w = make_uint4(bf16x2_to_f16x2(w.x), bf16x2_to_f16x2(w.y), bf16x2_to_f16x2(w.z), bf16x2_to_f16x2(w.w));
    return w;
}
// D = A B + D, and D = A B, m16n8k16 in f16 with 32-bit sums (not volatile: the compiler may order them)
__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// x within [-top, top]; a NaN of either stays what x is
__device__ __forceinline__ float within(float x, float top) { return x > top ? top : x < -top ? -top : x; }
template <int NG>
__device__ __forceinline__ void load_meta(uint32_t addr, uint32_t* m) {
    if constexpr (NG == 1) {
        asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(m[0]) : "r"(addr));
    } else if constexpr (NG == 2) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];\n" : "=r"(m[0]), "=r"(m[1]) : "r"(addr));
    } else {
#pragma unroll
        for (int i = 0; i < NG; i += 4)
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(m[i]), "=r"(m[i + 1]), "=r"(m[i + 2]), "=r"(m[i + 3])
                         : "r"(addr + 4 * i));
    }
}

template <int D, int NG>
__global__ void __launch_bounds__((I4Geom<D, NG>::THREADS), (I4Geom<D, NG>::CTAS)) rpa_int4_attn(const I4Params p) {
    using Gm = I4Geom<D, NG>;
    constexpr int NS = Gm::NS, KS = Gm::KS, CW = Gm::CW, C = D / 32, SUBS = 2;  // C: 16-byte chunks of a row of codes
    constexpr int CPG = C / NG;                                               // ... of a group
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ __align__(8) uint64_t full_bar[NS], empty_bar[NS], merge_bar, q_full, q_empty, q_shared;
    __shared__ __align__(16) int meta[NS][kMetaWords];
    __shared__ float red_ml[CW][R][2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const AttnParams& a = p.a;
    int* ctrl = a.ctrl;
    const uint64_t tmo = p.timeout_ns;
    const uint32_t ring0 = smem_u32(smem);
    const uint8_t* qbuf = smem + NS * Gm::STAGE;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(smem_u32(&full_bar[i]), 1);
            mbar_init(smem_u32(&empty_bar[i]), CW);
        }
        mbar_init(smem_u32(&merge_bar), CW);
        mbar_init(smem_u32(&q_full), 1);
        mbar_init(smem_u32(&q_empty), CW);
        mbar_init(smem_u32(&q_shared), CW);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_trigger();
    pdl_wait();  // the planner's items are complete from here on
    const int G = a.G, Hq = a.Hq, BR = p.BR, brs = p.brs, RB = BR * Gm::KB;

    if (warp == CW) {
        // =============================== producer ===============================
        if (p.stall == 1) return;
        const int ps = a.ps, runs = KS / BR;
        // K/V is read once, unless several blocks of query heads share it
        const uint64_t pol = p.blocks > 1 ? l2_policy_evict_last() : l2_policy_evict_first();
        int s = 0;
        uint32_t ph = 0, qph = 0;
        // An item, and the next one's description, which is fetched while this one's keys are on their way: its number, then its
        // unit, then its lengths, then its first page ids, each a stage after what it depends on.
        struct Work {
            Item item;
            int q_start, q_end, kl, lo, hi, nst0, nst, win0, win, win2;  // (page ids from win0 on, 64 of them)
        } cur, nxt;
        auto fetch_unit = [&](Work& x, int it) { x.item = item_at(a.units, it, a.unit_heads); };
        auto fetch_lengths = [&](Work& x) {
            x.q_start = a.cu_q_lens[x.item.seq];
            x.q_end = a.cu_q_lens[x.item.seq + 1];
            x.kl = a.kv_lens[x.item.seq];
        };
        auto fetch_pages = [&](Work& x) {
            // the unit's keys are those that any tile of the sequence sees: this tile's of them (none: a stage without keys,
            // whose item writes an empty partial)
            const int p_lo = x.kl - (x.q_end - x.q_start) + x.item.tok0, p_hi = p_lo + x.item.ntok - 1;
            x.lo = x.item.kv_begin;
            x.hi = x.item.kv_end;
            if (a.causal) x.hi = min(x.hi, p_hi + 1);
            if (a.has_window && (a.first == 0 || x.lo > a.first)) x.lo = max(x.lo, p_lo - a.window + 1);
            x.hi = max(x.hi, x.lo);
            const int key0 = x.lo & ~(BR - 1);
            x.nst0 = first_tiles(a, x.item, KS);
            x.nst = max(1, x.nst0 + (x.hi > x.lo ? (x.hi - key0 + KS - 1) / KS : 0));
            x.win0 = p.page.div(x.nst0 ? 0 : key0);
            const int* ids = a.page_indices + (size_t)x.item.seq * a.P + x.win0 + lane;
            x.win = (x.win0 + lane < a.P) ? ids[0] : 0;
            x.win2 = (x.win0 + 32 + lane < a.P) ? ids[32] : 0;
        };
        // the first item is the CTA's own, its unit on its way with the number of items (where there is none of that number, what
        // the list holds there is not used); the others come off a counter
        int it = blockIdx.x;
        if (it < p.most_items) fetch_unit(cur, it);
        const int ctas = min(ctrl[kDecCtas], (int)gridDim.x), n_items = it < ctas ? ctrl[a.item_count_word] : 0;
        bool ok = true;
        if (it < n_items) {
            fetch_lengths(cur);
            fetch_pages(cur);
        }
        while (ok && it < n_items) {
            int more = 0;
            if (lane == 0) more = ctas + atomicAdd(ctrl + a.counter_word, 1);
            const Item& item = cur.item;
            const int* ptab = a.page_indices + (size_t)item.seq * a.P;
            const int kvh = item.head / p.blocks;
            const int lo = cur.lo, hi = cur.hi, nst0 = cur.nst0, nst = cur.nst, key0 = lo & ~(BR - 1);
            const int p_lo = cur.kl - (cur.q_end - cur.q_start) + item.tok0, tok = cur.q_start + item.tok0;
            int win0 = cur.win0, win = cur.win, win2 = cur.win2, stage_of_next = 0;
            const int h0 = (item.head - kvh * p.blocks) * G, nh = min(G, p.heads - h0);  // its heads of the kv head's
            const uint32_t q_row = (uint32_t)(nh * D * 2);                             // bytes of a token's
            // Q, once the consumers have the last item's in registers
            if (!mbar_wait(smem_u32(&q_empty), qph ^ 1u, ctrl, tmo)) {
                ok = false;
                break;
            }
            qph ^= 1u;
            const uint32_t qfb = smem_u32(&q_full);
            if (lane == 0) mbar_arrive_expect_tx(qfb, (uint32_t)item.ntok * q_row);
            __syncwarp();
            if (lane < item.ntok)
                bulk_copy(ring0 + NS * Gm::STAGE + lane * (G * D * 2), a.q + ((size_t)(tok + lane) * Hq + kvh * p.heads + h0) * (D * 2), q_row,
                          qfb, pol);
            for (int st = 0; st < nst; ++st) {
                const bool fs = st < nst0;
                const int k_stage = fs ? st * KS : key0 + (st - nst0) * KS;
                const int kv_begin = fs ? 0 : lo, kv_end = fs ? a.first : hi;
                const int lp_last = p.page.div(max(k_stage, min(k_stage + KS, kv_end) - 1));
                if (lp_last - win0 >= 64) {
                    win0 = p.page.div(k_stage);
                    win = (win0 + lane < a.P) ? ptab[win0 + lane] : 0;
                    win2 = (win0 + 32 + lane < a.P) ? ptab[win0 + 32 + lane] : 0;
                }
                if (!mbar_wait(smem_u32(&empty_bar[s]), ph ^ 1u, ctrl, tmo)) {
                    ok = false;
                    break;
                }
                const uint32_t stage = ring0 + s * Gm::STAGE;
                // a lane takes a run of BR keys, and with runs of 4 keys another 32 runs on
                auto run_of = [&](int r, int& k0, int& lp, bool& want) {
                    k0 = k_stage + r * BR;
                    lp = p.page.div(k0);
                    const int i = lp - win0, x = __shfl_sync(0xffffffffu, win, i & 31), y = __shfl_sync(0xffffffffu, win2, i & 31);
                    want = r < runs && k0 < kv_end && k0 + BR > kv_begin;
                    return i < 32 ? x : y;
                };
                int k0[2], lp[2], pg[2];
                bool want[2] = {false, false};
                pg[0] = run_of(lane, k0[0], lp[0], want[0]);
                if (BR == 4) pg[1] = run_of(lane + 32, k0[1], lp[1], want[1]);
                bool good[2], bad = false;
                int n_issue = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    good[i] = want[i] && (unsigned)pg[i] < (unsigned)a.N;
                    bad |= want[i] && !good[i];
                    n_issue += __popc(__ballot_sync(0xffffffffu, good[i]));
                }
                if (__any_sync(0xffffffffu, bad)) {
                    // a page id outside [0, N): never dereferenced; its keys read as zero
                    if (lane == 0) set_status(ctrl, RPA_ERR_BAD_PAGE_INDEX);
                    for (int i = lane; i < Gm::STAGE / 16; i += 32)
                        reinterpret_cast<uint4*>(smem + s * Gm::STAGE)[i] = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                }
                // where the codes' chunks lie goes by a key's slot modulo 8: with runs of 4 keys, bit 2 of it for each run
                uint32_t swz = 0, swz2 = 0;
                if (BR == 4) {
                    swz = __ballot_sync(0xffffffffu, (k0[0] - lp[0] * ps) & 4);
                    swz2 = __ballot_sync(0xffffffffu, (k0[1] - lp[1] * ps) & 4);
                }
                if (lane == 0) {
                    int4* m = reinterpret_cast<int4*>(meta[s]);
                    m[0] = make_int4(k_stage, kv_begin, kv_end, nst - 1 - st);
                    m[1] = make_int4(p_lo, item.ntok, (int)swz, st == 0);
                    m[2] = make_int4(kvh * p.heads + h0, tok, item.part, nh);
                    if (BR == 4) m[3].x = (int)swz2;
                }
                __syncwarp();
                const uint32_t fb = smem_u32(&full_bar[s]);
                if (lane == 0) mbar_arrive_expect_tx(fb, (uint32_t)(n_issue * RB));
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!good[i]) continue;
                    const uint8_t* src = a.kv + ((size_t)pg[i] * a.Hkv + kvh) * p.block;
                    const uint32_t dst = stage + (lane + 32 * i) * RB;
                    if (BR == ps) {
                        bulk_copy(dst, src, RB, fb, pol);
                    } else {
                        const int r0 = k0[i] - lp[i] * ps;
                        bulk_copy(dst, src + r0 * (D / 2), BR * (D / 2), fb, pol);
                        bulk_copy(dst + BR * (D / 2), src + (size_t)(ps + r0) * (D / 2), BR * (D / 2), fb, pol);
                        bulk_copy(dst + BR * D, src + (size_t)ps * D + r0 * (NG * 4), BR * NG * 4, fb, pol);
                        bulk_copy(dst + BR * (D + NG * 4), src + (size_t)ps * D + (size_t)(ps + r0) * (NG * 4), BR * NG * 4, fb, pol);
                    }
                }
                if (++s == NS) {
                    s = 0;
                    ph ^= 1u;
                }
                if (stage_of_next == 0) more = __shfl_sync(0xffffffffu, more, 0);
                if (more < n_items) {
                    if (stage_of_next == 0) fetch_unit(nxt, more);
                    else if (stage_of_next == 1) fetch_lengths(nxt);
                    else if (stage_of_next == 2) fetch_pages(nxt);
                }
                ++stage_of_next;
            }
            if (!ok) break;
            it = more;
            if (it < n_items) {
                if (stage_of_next < 2) fetch_lengths(nxt);
                if (stage_of_next < 3) fetch_pages(nxt);
                cur = nxt;
            }
        }
        if (ok && !p.stall && mbar_wait(smem_u32(&empty_bar[s]), ph ^ 1u, ctrl, tmo)) {
            if (lane == 0) {
                meta[s][mLeft] = -1;
                mbar_arrive(smem_u32(&full_bar[s]));
            }
        } else {
            // gave up: let the copies already issued land before leaving
            drain_ring(full_bar, NS, s, ph, ctrl, tmo);
            drain_ring(&q_full, 1, 0, qph, ctrl, tmo);
        }
        return;
    }

    // =============================== consumers ===============================
    // ---- Thread (g = lane / 4, t = lane % 4) holds, of S^T, rows 2t and 2t + 1 of keys g and g + 8 of each 16; of O^T those rows
    // of channels 32 c + 4 g .. + 3.
    const int w = warp, g = lane >> 2, t = lane & 3;
    const uint32_t mb = smem_u32(&merge_bar);
    int s = 0;
    uint32_t ph = 0, mph = 0, qph = 0;
    uint32_t qf[Gm::QSH ? 1 : C][4];
    uint4* const q_ops = reinterpret_cast<uint4*>(smem + NS * Gm::STAGE + Gm::QB) + lane;  // chunk c's at 32 c
    float qs[2][NG];          // sums of q over a group, times 2^-20
    float o_acc[C][2][4];     // [.][i][0, 1]: channel 32 c + 4 g + 2 i, rows 2t, 2t + 1, times 2^-24; [2, 3]: and 16 times the next channel
    float psum[NG][4];        // sums of P (rows 2t, 2t + 1, twice)
    float zs[2][NG];          // sums of p (z + 8 s) over this thread's keys
    float m_r[2], l_r[2];
    int pos[2];
    constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u, kByte = 0x00ff00ffu;
    // Within a stage: this lane's row of codes for the matrix loads (of the first 16 keys), the (scale, zero) pairs of key g,
    // and how far on those of the next 16 keys, and of key g + 8, lie; the place of the row's chunk 0 (of matrices 2, 3: 1)
    const uint32_t row0 = (uint32_t)(((32 * w + (lane & 15)) >> brs) * RB + ((32 * w + (lane & 15)) & (BR - 1)) * (D / 2));
    const uint32_t pair0 = (uint32_t)(((32 * w + g) >> brs) * RB + BR * D + ((32 * w + g) & (BR - 1)) * (NG * 4));
    const uint32_t row16 = BR >= 32 ? 16 * (D / 2) : (16 >> brs) * RB, pair16 = BR >= 32 ? 16 * (NG * 4) : (16 >> brs) * RB;
    const uint32_t pair8 = BR >= 16 ? 8 * (NG * 4) : (8 >> brs) * RB;
    uint32_t sw[SUBS];
#pragma unroll
    for (int i = 0; i < SUBS; ++i) sw[i] = ((lane >> 4) ^ ((lane & 7) * D / 256 & (C - 1))) << 4;
    for (;;) {
        if (!mbar_wait(smem_u32(&full_bar[s]), ph, ctrl, tmo)) return;
        const int4 m0 = *reinterpret_cast<const int4*>(&meta[s][mKey0]), m1 = *reinterpret_cast<const int4*>(&meta[s][mPos]);
        const int kv_begin = m0.y, kv_end = m0.z, left = m0.w;  // left: the item's stages behind this one (-1: no more items)
        if (left < 0) return;
        const int p_lo = m1.x, ntok = m1.y;                     // p_lo: position of the tile's first token
        if (m1.w) {
            // row g of Q: channels 32 c + 8 t .. + 7 of each chunk, paired as the masks pair the codes
            const bool live = g < ntok * G && g % G < meta[s][mHeads];
            if (!mbar_wait(smem_u32(&q_full), qph, ctrl, tmo)) return;
            qph ^= 1u;
            float sum[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) sum[i] = 0.f;
            uint4 x[C];
#pragma unroll
            for (int c = 0; c < C; ++c) x[c] = live ? load_q8(qbuf, g * D + 8 * t + 32 * c, a.q_f16 == 0) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                // channels 0, 4; 2, 6; 1, 5; 3, 7
                const uint4 f = make_uint4(__byte_perm(x[c].x, x[c].z, 0x5410), __byte_perm(x[c].y, x[c].w, 0x5410),
                                           __byte_perm(x[c].x, x[c].z, 0x7632), __byte_perm(x[c].y, x[c].w, 0x7632));
                if constexpr (Gm::QSH) {
                    if (c % CW == w) q_ops[32 * c] = f;  // (the last item's are free: its merge has seen every warp)
                } else {
                    qf[c][0] = f.x; qf[c][1] = f.y; qf[c][2] = f.z; qf[c][3] = f.w;
                }
                const uint32_t xs[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = f16x2_to_f32x2(xs[i]);
                    sum[c / CPG] += f.x + f.y;
                }
            }
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
                sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
#pragma unroll
                for (int ri = 0; ri < 2; ++ri) {
                    qs[ri][i] = __shfl_sync(0xffffffffu, sum[i], 4 * (2 * t + ri)) * 9.5367431640625e-7f;
                    zs[ri][i] = 0.f;
                }
                psum[i][0] = psum[i][1] = psum[i][2] = psum[i][3] = 0.f;
            }
#pragma unroll
            for (int ri = 0; ri < 2; ++ri) {
                m_r[ri] = -INFINITY;
                l_r[ri] = 0.f;
                pos[ri] = p_lo + (2 * t + ri) / G;
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) o_acc[c][i][0] = o_acc[c][i][1] = o_acc[c][i][2] = o_acc[c][i][3] = 0.f;
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&q_empty));
            if constexpr (Gm::QSH) {
                if (lane == 0) mbar_arrive(smem_u32(&q_shared));
                if (!mbar_wait(smem_u32(&q_shared), qph ^ 1u, ctrl, tmo)) return;
            }
        }
        const int kw = m0.x + 32 * w;  // this warp's 32 keys
        if (kw < kv_end && kw + 32 > kv_begin) {
            const uint32_t swz = (uint32_t)m1.z, stage = ring0 + s * Gm::STAGE;
            const bool need_mask = kw < kv_begin || kw + 32 > kv_end || (a.causal && kw + 31 > p_lo) ||
                                   (a.has_window && kw <= p_lo + ntok - 1 - a.window);
            if (BR == 4) {  // where the chunks lie goes by the slot modulo 8, which runs of 4 keys start at 0 or 4
                const uint32_t mine = (w < 4 ? swz : (uint32_t)meta[s][mSwz2]) >> (8 * (w & 3));
#pragma unroll
                for (int i = 0; i < SUBS; ++i) {
                    const uint32_t r8 = (mine >> (4 * i + ((lane & 15) >> 2)) & 1u) * 4 + (lane & 3);
                    sw[i] = ((lane >> 4) ^ (r8 * D / 256 & (C - 1))) << 4;
                }
            }
            uint64_t x[SUBS][2];    // logits of rows 2t, 2t + 1: key g, key g + 8
            uint32_t vm[SUBS][2][NG];
#pragma unroll
            for (int sub = 0; sub < SUBS; ++sub) {
                const uint32_t row = stage + row0 + (sub ? row16 : 0u), at = stage + pair0 + (sub ? pair16 : 0u);
                uint32_t km[2][NG];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    load_meta<NG>(at + (h ? pair8 : 0u), km[h]);
                    load_meta<NG>(at + (h ? pair8 : 0u) + BR * (NG * 4), vm[sub][h]);
                }
                float e[4], o[4];
                uint32_t kf[C / 2][4];
#pragma unroll
                for (int c = 0; c < C; c += 2)
                    ldsm_x4(row + ((uint32_t)(c << 4) ^ sw[sub]), kf[c / 2][0], kf[c / 2][1], kf[c / 2][2], kf[c / 2][3]);
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    const uint32_t* f = kf[c / 2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int cc = c + h;
                        const uint32_t u0 = f[2 * h], u1 = f[2 * h + 1], v0 = u0 >> 8, v1 = u1 >> 8;
                        const uint32_t ae[4] = {u0 & kLow, u1 & kLow, v0 & kLow, v1 & kLow};
                        const uint32_t ao[4] = {u0 & kHigh, u1 & kHigh, v0 & kHigh, v1 & kHigh};
                        uint4 qv;
                        if constexpr (Gm::QSH) qv = q_ops[32 * cc];
                        else qv = make_uint4(qf[cc][0], qf[cc][1], qf[cc][2], qf[cc][3]);
                        if (cc % CPG == 0) {
                            mma_first(e, ae, qv.x, qv.y);
                            mma_first(o, ao, qv.z, qv.w);
                        } else {
                            mma(e, ae, qv.x, qv.y);
                            mma(o, ao, qv.z, qv.w);
                        }
                        if ((cc + 1) % CPG == 0) {
                            const int gi = cc / CPG;
#pragma unroll
                            for (int hk = 0; hk < 2; ++hk) {
                                const float2 sz = f16x2_to_f32x2(km[hk][gi]);
                                const uint64_t ss = f32x2(sz.x, sz.x), zz = f32x2(sz.y, sz.y), q2 = f32x2(qs[0][gi], qs[1][gi]);
                                const uint64_t raw = ffma2(f32x2(e[2 * hk], e[2 * hk + 1]), f32x2(16.f, 16.f), f32x2(o[2 * hk], o[2 * hk + 1]));
                                x[sub][hk] = ffma2(ss, raw, gi == 0 ? fmul2(zz, q2) : ffma2(zz, q2, x[sub][hk]));
                            }
                        }
                    }
                }
            }
            // the first 16 keys' V, on its way during the softmax
            uint32_t vf[C / 2][4];
            auto load_v = [&](int sub) {
                const uint32_t row = stage + row0 + (sub ? row16 : 0u) + BR * (D / 2);
#pragma unroll
                for (int c = 0; c < C; c += 2)
                    ldsm_x4_t(row + ((uint32_t)(c << 4) ^ sw[sub]), vf[c / 2][0], vf[c / 2][1], vf[c / 2][2], vf[c / 2][3]);
            };
            if constexpr (D < 256) load_v(0);
            // ---- scale or soft cap (log2 domain), then masks
            if (a.has_cap) {
                const float ce = a.cap_exp * 1048576.f, cl = a.cap_log2;
#pragma unroll
                for (int i = 0; i < 2 * SUBS; ++i) {
                    float y[2];
                    f32x2_split(x[i / 2][i % 2], y[0], y[1]);
#pragma unroll
                    for (int ri = 0; ri < 2; ++ri) y[ri] = cl - 2.f * cl * rcp_approx(1.f + ex2(y[ri] * ce));
                    x[i / 2][i % 2] = f32x2(y[0], y[1]);
                }
            } else {
                const float qk = a.qk_log2 * 1048576.f;
                const uint64_t qk2 = f32x2(qk, qk);
#pragma unroll
                for (int i = 0; i < 2 * SUBS; ++i) x[i / 2][i % 2] = fmul2(x[i / 2][i % 2], qk2);
            }
            if (need_mask) {
#pragma unroll
                for (int sub = 0; sub < SUBS; ++sub)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = kw + 16 * sub + g + 8 * h;
                        const bool in = j >= kv_begin && j < kv_end;
                        if (!in) {  // the scales of keys outside the range may hold any bits
#pragma unroll
                            for (int i = 0; i < NG; ++i) vm[sub][h][i] = 0u;
                        }
                        float y[2];
                        f32x2_split(x[sub][h], y[0], y[1]);
#pragma unroll
                        for (int ri = 0; ri < 2; ++ri) {
                            const bool okk = in && (!a.causal || j <= pos[ri]) && (!a.has_window || j > pos[ri] - a.window || j < a.first);
                            y[ri] = okk ? y[ri] : -INFINITY;
                        }
                        x[sub][h] = f32x2(y[0], y[1]);
                    }
            }
            // ---- the running maximum moves only when a key outgrows it (by 2^2): each lane looks at its own keys, and only
            // then are the rows' maxima formed across lanes
            float mx[2];
            {
                float y[2][2 * SUBS];
#pragma unroll
                for (int i = 0; i < 2 * SUBS; ++i) f32x2_split(x[i / 2][i % 2], y[0][i], y[1][i]);
#pragma unroll
                for (int ri = 0; ri < 2; ++ri) {
                    mx[ri] = fmaxf(y[ri][0], y[ri][1]);
                    if constexpr (SUBS == 2) mx[ri] = fmax3(mx[ri], y[ri][2], y[ri][3]);
                }
            }
            if (__any_sync(0xffffffffu, mx[0] > m_r[0] + kRescale || mx[1] > m_r[1] + kRescale)) {
#pragma unroll
                for (int ri = 0; ri < 2; ++ri) {
                    float v = mx[ri];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    const float m_new = fmaxf(m_r[ri], v);
                    const float alpha = m_r[ri] == -INFINITY ? 0.f : ex2(m_r[ri] - m_new);
                    m_r[ri] = m_new;
                    l_r[ri] *= alpha;
#pragma unroll
                    for (int i = 0; i < NG; ++i) {
                        zs[ri][i] *= alpha;
                        psum[i][ri] *= alpha;
                    }
#pragma unroll
                    for (int c = 0; c < C; ++c)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            o_acc[c][i][ri] *= alpha;
                            o_acc[c][i][ri + 2] *= alpha;
                        }
                }
            }
            {
                const uint64_t nb = f32x2(m_r[0] == -INFINITY ? 0.f : -m_r[0], m_r[1] == -INFINITY ? 0.f : -m_r[1]);
                uint64_t l2 = f32x2(l_r[0], l_r[1]);
#pragma unroll
                for (int i = 0; i < 2 * SUBS; ++i) {
                    float y[2];
                    f32x2_split(fadd2(x[i / 2][i % 2], nb), y[0], y[1]);
                    x[i / 2][i % 2] = f32x2(ex2(y[0]), ex2(y[1]));
                    l2 = fadd2(l2, x[i / 2][i % 2]);
                }
                f32x2_split(l2, l_r[0], l_r[1]);
            }
            // ---- O^T += V^T P^T, group by group
#pragma unroll
            for (int sub = 0; sub < SUBS; ++sub) {
                uint32_t pb[2];
                if (sub || D == 256) load_v(sub);
#pragma unroll
                for (int c = 0; c < C; c += 2) {
                    const uint32_t* f = vf[c / 2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int cc = c + h, gi = cc / CPG;
                        if (cc % CPG == 0) {
                            const float2 a0 = f16x2_to_f32x2(vm[sub][0][gi]), a1 = f16x2_to_f32x2(vm[sub][1][gi]);
                            const float mid0 = fmaf(8.f, a0.x, a0.y), mid1 = fmaf(8.f, a1.x, a1.y);
                            f32x2_split(ffma2(x[sub][0], f32x2(mid0, mid0), ffma2(x[sub][1], f32x2(mid1, mid1), f32x2(zs[0][gi], zs[1][gi]))),
                                        zs[0][gi], zs[1][gi]);
                            float b0, b1, b2, b3;
                            f32x2_split(fmul2(x[sub][0], f32x2(a0.x, a0.x)), b0, b1);
                            f32x2_split(fmul2(x[sub][1], f32x2(a1.x, a1.x)), b2, b3);
                            pb[0] = transposed(pack2<true>(b0, b1));
                            pb[1] = transposed(pack2<true>(b2, b3));
                            constexpr uint32_t one = 0x3c003c00u;
                            const uint32_t ones[4] = {one, one, one, one};
                            mma(psum[gi], ones, pb[0], pb[1]);
                        }
                        const uint32_t u0 = f[2 * h] & kByte, u1 = f[2 * h + 1] & kByte;
                        const uint32_t v0 = __byte_perm(f[2 * h], 0u, 0x4341), v1 = __byte_perm(f[2 * h + 1], 0u, 0x4341);
                        const uint32_t a0[4] = {u0 & kLow, u0, u1 & kLow, u1};
                        const uint32_t a1[4] = {v0 & kLow, v0, v1 & kLow, v1};
                        mma(o_acc[cc][0], a0, pb[0], pb[1]);
                        mma(o_acc[cc][1], a1, pb[0], pb[1]);
                    }
                }
            }
        }
        const int4 m2 = *reinterpret_cast<const int4*>(&meta[s][mHead]);
        __syncwarp();
        const uint32_t slot = smem_u32(&empty_bar[s]);
        float* red_o = reinterpret_cast<float*>(smem + s * Gm::STAGE);  // [CW][R][LD]
        if (++s == NS) {
            s = 0;
            ph ^= 1u;
        }
        if (left > 0) {
            if (lane == 0) mbar_arrive(slot);
            continue;
        }
        // ---- the item's end: merge the warps' partials through its last stage
        if (lane == 0) mbar_arrive(mb);  // A: every warp is done with the stage
        if (!mbar_wait(mb, mph, ctrl, tmo)) return;
        mph ^= 1u;
#pragma unroll
        for (int ri = 0; ri < 2; ++ri) {
            float l = l_r[ri];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int r = 2 * t + ri;
            if (g == 0) {
                red_ml[w][r][0] = m_r[ri];
                red_ml[w][r][1] = l;
            }
            float add[NG];
#pragma unroll
            for (int i = 0; i < NG; ++i) {
                float z = zs[ri][i];
                z += __shfl_xor_sync(0xffffffffu, z, 4);
                z += __shfl_xor_sync(0xffffffffu, z, 8);
                z += __shfl_xor_sync(0xffffffffu, z, 16);
                add[i] = fmaf(-8.f, psum[i][ri], z);
            }
            float* out = red_o + (w * R + r) * Gm::LD + 4 * g;
#pragma unroll
            for (int c = 0; c < C; ++c)
                *reinterpret_cast<float4*>(out + 32 * c) =
                    make_float4(fmaf(o_acc[c][0][ri], 16777216.f, add[c / CPG]), fmaf(o_acc[c][0][ri + 2] - o_acc[c][0][ri], 1048576.f, add[c / CPG]),
                                fmaf(o_acc[c][1][ri], 16777216.f, add[c / CPG]), fmaf(o_acc[c][1][ri + 2] - o_acc[c][1][ri], 1048576.f, add[c / CPG]));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(mb);  // B: every partial is in shared memory
        if (!mbar_wait(mb, mph, ctrl, tmo)) return;
        mph ^= 1u;
        const int rows = ntok * G, part = m2.z;
        for (int e = w * 32 + lane; e < rows * (D / 4); e += CW * 32) {
            const int r = e / (D / 4), c = (e % (D / 4)) * 4, hr = r % G;
            if (hr >= m2.w) continue;  // (a block of fewer heads)
            float M = -INFINITY;
#pragma unroll
            for (int i = 0; i < CW; ++i) M = fmaxf(M, red_ml[i][r][0]);
            // (nothing is visible, or every visible logit is a NaN, which no maximum takes: L is 0, or the NaN that a warp's l is)
            const float base = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < CW; ++i) {
                const float sc = ex2(red_ml[i][r][0] - base);
                L += sc * red_ml[i][r][1];
                if (M != -INFINITY) {
                    const float4 v = *reinterpret_cast<const float4*>(red_o + (i * R + r) * Gm::LD + c);
                    o.x += sc * v.x;
                    o.y += sc * v.y;
                    o.z += sc * v.z;
                    o.w += sc * v.w;
                }
            }
            const float top = kMostHalf * L;  // values end at +-65504 here as they do in f16 rows, and means of them do, whatever P's rounding adds
            o = make_float4(within(o.x, top), within(o.y, top), within(o.z, top), within(o.w, top));
            if (part < 0) {
                const int tok = m2.y + r / G, qh = m2.x + hr;
                L = add_sink(L, a.sinks, qh, M);
                const float inv = L > 0.f ? a.v_scale / L : 0.f * L;  // (a NaN stays one)
                store_o4(a.o, ((size_t)tok * Hq + qh) * D + c, o.x * inv, o.y * inv, o.z * inv, o.w * inv, a.odt);
            } else {
                *reinterpret_cast<float4*>(a.part_o + ((size_t)part * R + r) * D + c) = o;
                if (c == 0) *reinterpret_cast<float2*>(a.part_ml + ((size_t)part * R + r) * 2) = make_float2(M, L);
            }
        }
        fence_proxy_async_smem();  // the stage will be refilled by bulk copies
        __syncwarp();
        if (lane == 0) mbar_arrive(slot);
    }
}

// ---------------------------------------------------------------- long prompts: the cache's rows in f16
struct UnfoldParams {
    const uint8_t* kv;
    uint8_t* rows;       // [room pages][64][2 Hkv][D] f16
    int* table;          // [max_num_seqs][P64]
    const int *kv_lens, *page_indices, *cu, *vbase;
    const uint8_t* q;    // bf16, rounded to f16 into qbuf (where that is set)
    uint8_t* qbuf;
    int* ctrl;
    int S, T, Hq, Hkv, D, ps, P, N, P64, group;
    int has_window, window, first;
};

constexpr int kUnfoldThreads = 256, kUnfoldCtas = 5;

// V's rows end one step in front of f16's last value: a mean of them with P rounded (by 2^-11 at most) is then none past it
constexpr float kMostRow = 65472.f;
__device__ __forceinline__ void saturate_row(float* f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i] = within(f[i], kMostRow);
}

__global__ void __launch_bounds__(kUnfoldThreads, kUnfoldCtas) rpa_int4_unfold(const UnfoldParams p) {
    pdl_trigger();
    pdl_wait();
    if (p.ctrl[kNumPfItems] == 0) return;
    const int tid = threadIdx.x, lane = tid & 31;
    const int total = p.vbase[p.S], per_row = p.D / 16;
    // up to kSeqs sequences' first pages, query tokens and keys (beside more a warp searches a task's sequence)
    constexpr int kSeqs = 512;
    __shared__ int s_base[kSeqs + 1], s_ql[kSeqs], s_kl[kSeqs], s_seq;
    const bool few = p.S <= kSeqs;
    if (few) {
        for (int i = tid; i < p.S; i += kUnfoldThreads) {
            s_base[i] = p.vbase[i];
            s_ql[i] = p.cu[i + 1] - p.cu[i];
            s_kl[i] = p.kv_lens[i];
        }
        __syncthreads();
    }
    // a task: 64 keys of one kv head
    for (int task = blockIdx.x; task < total * p.Hkv; task += gridDim.x) {
        const int v = task / p.Hkv, h = task - v * p.Hkv;
        int s = 0;
        if (few) {
            s = last_start(s_base, p.S, v);  // the last sequence whose pages start at or before v
        } else {
            __syncthreads();
            if (tid < 32) {
                const int x = find_seq(p.vbase, p.S, v, lane);
                if (lane == 0) s_seq = x;
            }
            __syncthreads();
            s = s_seq;
            if (s < 0) continue;  // (not reached: vbase covers the pages)
        }
        const int base = few ? s_base[s] : p.vbase[s];
        const int ql = few ? s_ql[s] : p.cu[s + 1] - p.cu[s], kl = few ? s_kl[s] : p.kv_lens[s];
        int lo = p.has_window ? max(0, kl - ql - p.window + 1) : 0;
        if (lo <= p.first) lo = 0;
        const int nf = lo > 0 ? (p.first + 63) / 64 : 0, at = v - base;
        const int page64 = at < nf ? at : lo / 64 + at - nf;
        if (h == 0 && tid == 0) p.table[(size_t)s * p.P64 + page64] = v;
        // a thread takes one unit of 16 channels of K and V of a key, kFly keys in flight
        const int step = kUnfoldThreads / per_row, place = tid % per_row;
        constexpr int kFly = 2;
        for (int slot0 = tid / per_row; slot0 < 64; slot0 += kFly * step) {
            uint2 codes[kFly][2];
            uint32_t pairs[kFly][2];
            bool good[kFly];
#pragma unroll
            for (int b = 0; b < kFly; ++b) {
                const int slot = slot0 + b * step, j = page64 * 64 + slot;
                good[b] = false;
                if (slot >= 64 || j >= kl) continue;  // (rows past the last are masked, whatever they hold)
                const int pg = p.page_indices[(size_t)s * p.P + j / p.ps], ks = j % p.ps;
                good[b] = (unsigned)pg < (unsigned)p.N;
                if (!good[b]) {
                    // (pages that no token of the call sees are not checked: a page of 64 may be wider than the band)
                    if (j >= lo || j < p.first) set_status(p.ctrl, RPA_ERR_BAD_PAGE_INDEX);
                    continue;
                }
                const uint8_t* block = p.kv + ((size_t)pg * p.Hkv + h) * ((size_t)p.ps * int4_key_bytes(p.D, p.group));
#pragma unroll
                for (int is_v = 0; is_v < 2; ++is_v) {
                    const uint32_t line = (uint32_t)(is_v ? p.ps : 0) + ks;
                    codes[b][is_v] = *reinterpret_cast<const uint2*>(block + (size_t)line * (p.D / 2) + int4_chunk(place / 2, ks, p.D) * 16 + (place & 1) * 8);
                    pairs[b][is_v] = reinterpret_cast<const uint32_t*>(block + (size_t)p.ps * p.D)[(size_t)line * (p.D / p.group) + 16 * place / p.group];
                }
            }
#pragma unroll
            for (int b = 0; b < kFly; ++b) {
                const int slot = slot0 + b * step;
                if (slot >= 64 || page64 * 64 + slot >= kl) continue;
#pragma unroll
                for (int is_v = 0; is_v < 2; ++is_v) {
                    uint32_t out[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (good[b]) {
                        const float2 sz = f16x2_to_f32x2(pairs[b][is_v]);
                        float f[16];
                        int4_values(codes[b][is_v], sz, f);
                        if (!is_v) int4_saturate(sz, f);
                        else if (fmaxf(fabsf(sz.y), fmaf(15.f, sz.x, sz.y)) > kMostRow) saturate_row(f);
#pragma unroll
                        for (int k = 0; k < 8; ++k) out[k] = pack2<true>(f[2 * k], f[2 * k + 1]);
                    }
                    store_32(p.rows + ((((size_t)v * 64 + slot) * 2 * p.Hkv + 2 * h + is_v) * p.D + 16 * place) * 2, out);
                }
            }
        }
    }
    if (p.qbuf) {
        const size_t n = (size_t)p.T * p.Hq * p.D / 8;
        for (size_t i = (size_t)blockIdx.x * kUnfoldThreads + tid; i < n; i += (size_t)gridDim.x * kUnfoldThreads)
            reinterpret_cast<uint4*>(p.qbuf)[i] = load_q8(p.q, i * 8, 1);
    }
}

template <int D, int NG>
struct I4Kern {
    using Gm = I4Geom<D, NG>;
    static cudaError_t prepare(int* bps) {
        cudaError_t e = cudaFuncSetAttribute(rpa_int4_attn<D, NG>, cudaFuncAttributeMaxDynamicSharedMemorySize, Gm::SMEM);
        if (e != cudaSuccess) return e;
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(bps, rpa_int4_attn<D, NG>, Gm::THREADS, Gm::SMEM);
    }
    static cudaError_t launch(const I4Params& p, const Launch& l) {
        return launch_pdl(rpa_int4_attn<D, NG>, l.grid, Gm::THREADS, Gm::SMEM, l.stream, p);
    }
};

template <typename Op>
cudaError_t i4_dispatch(int D, int group, Op op) {
    if (D == 64) return group == 32 ? op(I4Kern<64, 2>{}) : group == 64 ? op(I4Kern<64, 1>{}) : cudaErrorInvalidValue;
    if (D == 128) return group == 32 ? op(I4Kern<128, 4>{}) : group == 64 ? op(I4Kern<128, 2>{}) : op(I4Kern<128, 1>{});
    if (D == 256) return group == 32 ? op(I4Kern<256, 8>{}) : group == 64 ? op(I4Kern<256, 4>{}) : op(I4Kern<256, 2>{});
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t int4_prepare(int D, int group, int* bps) {
    return i4_dispatch(D, group, [&](auto k) { return decltype(k)::prepare(bps); });
}

int enqueue_int4(const RpaCfg& c, const KernelSet& ks, const Workspace& ws, MapCache* maps, const AttnParams& a, int num_seqs,
                 const EnqueueOpts& eo) {
    cudaStream_t st = eo.st;
    auto rec = [&](int k) { return !eo.ev[k] || cudaEventRecord(eo.ev[k], st) == cudaSuccess; };
    const bool has_q = c.num_q_tokens > 0;
    // (prompts first: where there are none, these two end while the direct kernel is being launched, not after it)
    if (!rec(kEvPfStart)) return RPA_ERR_CUDA;
    if (has_q && ks.room_pages > 0) {
        UnfoldParams u;
        u.kv = a.kv;
        u.rows = ws.room;
        u.table = ws.room_table;
        u.kv_lens = a.kv_lens;
        u.page_indices = a.page_indices;
        u.cu = a.cu_q_lens;
        u.vbase = ws.vbase;
        u.q = a.q;
        u.qbuf = ks.q_conv ? nullptr : ws.qbuf;  // (q of 32 bits is there already)
        u.ctrl = ws.ctrl;
        u.S = num_seqs;
        u.T = (int)c.num_q_tokens;
        u.Hq = a.Hq;
        u.Hkv = a.Hkv;
        u.D = ks.D;
        u.ps = a.ps;
        u.P = a.P;
        u.N = a.N;
        u.P64 = ks.P64;
        u.group = ks.group;
        u.has_window = a.has_window;
        u.window = a.window;
        u.first = a.first;
        if (launch_pdl(rpa_int4_unfold, ks.sms * kUnfoldCtas, kUnfoldThreads, 0, st, u) != cudaSuccess) return RPA_ERR_CUDA;
        const void* q16 = u.qbuf ? ws.qbuf : a.q;
        if (maps->kv_ptr != ws.room) {
            if ((ks.tc8 ? encode_kv_map_heads(&maps->kv_pf, ws.room, ks.room_pages, 64, 2 * a.Hkv, ks.D, 64)
                        : encode_kv_map(&maps->kv_pf, ws.room, 0, ks.room_pages, 64, a.Hkv, ks.D, 64)) != 0) {
                maps->kv_ptr = nullptr;
                return RPA_ERR_INVALID_ARG;
            }
            maps->kv_ptr = ws.room;
        }
        if (maps->q_ptr != q16) {
            if (encode_q_map(&maps->q_pf, q16, c.num_q_tokens, a.Hq, ks.D, ks.G, kTcRows / ks.G) != 0) {
                maps->q_ptr = nullptr;
                return RPA_ERR_INVALID_ARG;
            }
            maps->q_ptr = q16;
        }
        TcParams tp;
        tp.a = a;
        tp.a.q = static_cast<const uint8_t*>(q16);
        tp.a.kv = ws.room;
        tp.a.page_indices = ws.room_table;
        tp.a.G = ks.G;
        tp.a.P = ks.P64;
        tp.a.ps = 64;
        tp.a.N = ks.room_pages;
        tp.a.units = ws.pf_units;
        tp.a.unit_heads = a.Hkv;
        tp.a.item_count_word = kNumPfItems;
        tp.a.counter_word = kPfCounter;
        tp.BR = 64;
        tp.Tq = ks.pf_tokens;
        tp.timeout_ns = eo.timeout_ns;
        const Launch l{ks.sms * ks.pf_bps, st};
        if ((ks.tc8 ? launch_prefill_tc8(maps->kv_pf, maps->q_pf, tp, KT_F16, l) : launch_prefill_tc(maps->kv_pf, maps->q_pf, tp, KT_F16, l)) !=
            cudaSuccess)
            return RPA_ERR_CUDA;
    }
    if (!rec(kEvPfEnd) || !rec(kEvDecStart)) return RPA_ERR_CUDA;
    if (has_q) {
        I4Params p;
        p.a = a;
        p.a.units = ws.dec_units;
        p.a.item_count_word = kNumDecItems;
        p.a.counter_word = kDecCounter;
        p.heads = ks.G;
        p.blocks = ks.Hp / (int)c.num_kv_heads;
        p.BR = int4_warps(ks.D) % 4 ? 32 : 128;  // runs divide a stage, of 32 keys a warp
        while (c.page_size % p.BR) p.BR >>= 1;
        p.brs = 0;
        while ((1 << p.brs) < p.BR) ++p.brs;
        p.block = (uint32_t)(c.page_size * int4_key_bytes(ks.D, ks.group));
        p.page.set((uint32_t)c.page_size);
        p.most_items = ks.max_dec_units * a.unit_heads;
        p.stall = eo.debug_stall;
        p.timeout_ns = eo.timeout_ns;
        if (i4_dispatch(ks.D, ks.group, [&](auto k) { return decltype(k)::launch(p, Launch{ks.sms * ks.dec_bps, st}); }) !=
            cudaSuccess)
            return RPA_ERR_CUDA;
    }
    return rec(kEvDecEnd) ? RPA_OK : RPA_ERR_CUDA;
}

}  // namespace rpa
