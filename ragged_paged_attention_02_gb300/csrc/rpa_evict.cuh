// rpa_evict.cuh -- parameters shared by the eviction kernels and their host side.
#pragma once

#include "rpa_internal.cuh"

namespace rpa {

// j / d for 0 <= j < 2^31 by one 32-bit high product (T. Granlund and P. L. Montgomery, Division by Invariant Integers
// using Multiplication, 1994): with l = ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1,
// j / d = (umulhi(m, j) + j) >> l (the sum stays below 2^32).
struct FastDiv {
    uint32_t d, m, l;
    void set(uint32_t div) {
        d = div;
        l = 0;
        while (((uint64_t)1 << l) < div) ++l;
        m = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << l) - div)) / div) + 1u;
    }
#ifdef __CUDACC__
    __device__ __forceinline__ int div(int j) const { return (int)((__umulhi(m, (uint32_t)j) + (uint32_t)j) >> l); }
#endif
};

// ---------------------------------------------------------------- accumulated weights
constexpr int kWeighRows = 16;     // query rows (tokens x heads of a group) of a block
constexpr int kWeighAlign = 128;   // pieces are multiples of this many keys
constexpr int kWeighKeys = 128;    // keys of a weigh item that reads logits back
constexpr int kWeighThreads = 128;

struct WeighParams {
    const uint8_t* q;        // in the MMA operand type, or bf16 with q_bf16
    const uint8_t* kv;
    const int *kv_lens, *page_indices, *cu;
    float* scores;
    int S, T, Hq, Hkv, G, D, ps, P, N;
    int causal, has_window, window, has_cap;
    int q_bf16;              // 8-bit K/V: q holds bf16, rounded to f16 as it is loaded
    float qk_log2;           // sm_scale * k_scale * log2(e)
    float cap_arg;           // sm_scale * k_scale / cap
    float cap_log2;          // cap * log2(e)
    const float* sinks;
    FastDiv page, group;
    int max_pieces;          // most pieces of a sequence
    int item_keys;           // keys of a weigh item that computes them again
    int ctas;                // of the stats kernel (all resident)
    int weigh_warps;         // of the weigh kernel
    int BR, br_shift;        // keys of a copied page run: gcd(page_size, 64), and its log2
    uint32_t all_runs;       // a bit for each run of 64 keys
    long long max_logits;    // floats the logit buffer holds
    // workspace
    int* status;             // sticky
    int* ctrl;               // [0] stat items, [1] weigh items, [2] stat items taken, [3] kv heads of a weigh item
    int* stat0;              // [S + 1] first stat item of a sequence
    int* item0;              // [S + 1] first weigh item
    int* block0;             // [S + 1] first row block (counting kv heads)
    long long* logit0;       // [S] first float of the sequence's logits, or -1: they are computed again
    int* done;               // [blocks] warps of a row block whose statistics are out
    float2* part;            // [blocks, max_pieces, 4 warps, kWeighRows] maximum (log2) and sum
    float* stat;             // [blocks, kWeighRows] maximum + log2 of the sum; infinite: nothing is seen
    float* logits;
};

// ---------------------------------------------------------------- compaction
struct CompactParams {
    uint8_t* kv;
    float* scores;
    const int *kv_lens, *page_indices, *new_pages;
    int* new_kv_lens;
    int* list;               // [S, Hkv, budget] kept slots (the caller's array or the workspace's)
    int fill;                // write -1 behind a list's end
    int* seq_n;              // [S] kept keys, or -1: bad lengths
    int* seq_order;          // [S] 1: rows move onto pages that hold other kept rows, in order then
    int* status;
    int S, Hkv, ps, P, N;
    int vec_shift;           // log2 of the 16-byte vectors of a row: K and V of one head in a slot
    int budget, protect, recent;
    int cluster;             // CTAs of a select cluster
    int move_cluster;        // CTAs of a move cluster
    int cached;              // scores a CTA of it keeps in shared memory
    FastDiv page;
};

// host launchers
// resident CTAs an SM of the stats kernel and the weigh kernel
cudaError_t weigh_prepare(int D, int kt, int* stats, int* weigh);
cudaError_t launch_weigh(const CUtensorMap& kmap, const WeighParams& p, int kt, int grid_weigh, cudaStream_t st);
cudaError_t compact_prepare(int64_t units, int max_keys, int sms, int* cluster, int* move_cluster, int* cached);
cudaError_t launch_compact(const CompactParams& p, int sms, cudaStream_t st);

}  // namespace rpa
