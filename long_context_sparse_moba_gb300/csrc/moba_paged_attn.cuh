// moba_paged_attn.cuh -- what the kernels of the attention over a paged cache
// share: the call's arguments, its entries (a tile of a sequence's query rows on
// one kv head) and the scratch.
#pragma once

#include <cuda_fp16.h>

#include "moba_paged.cuh"

namespace moba {
namespace paged {

constexpr int kTile = 64;        // keys per tile
constexpr int kMaxRows = 64;     // query rows of an entry at most
constexpr int kJobRows = 256;    // query rows of a job of the tcgen05 kernel
constexpr int kBigStart = 3;     // key tiles that the start of a span's job counts as
constexpr int kSelBad = -2;
constexpr int kMaxBlocks = 65536;  // blocks of a sequence where blocks are selected

// A tile of rows (numbered token * G + head) with the keys [key0, key_end) of sequence b's
// pages, those of a prefix whole, else each row's up to its position, its token + pdelta.
// A sequence's own span (with the keys from key0 on) names its group's: the group's first
// row, and where its spans begin among those of groups, << 1 | whether they are big.
struct alignas(16) Span {
    int row0, nrows;
    int b, full;
    int key0, key_end;
    int pdelta, pad;
    int group_row, group_span;
    int pads[2];
};
// Of the big spans [0] and the small ones [1], sequences' own before those of groups.
struct alignas(16) SpanHead {
    long long units[2];  // of all of them, times the kv heads
    int spans[2], own[2];
    int taken, pad[3];   // runs of small spans that have been taken
    unsigned long long ready, pads;  // the call's token once the plan is made; 0 again when the call ends
};

struct Attn {
    Cache c;
    const __nv_bfloat16 *q, *k, *v;
    const float *kbar;
    __nv_bfloat16 *out;
    float *lse;
    int32_t *idx;  // or nullptr
    int Hq, G, D, topk, km1;
    bool dense;     // topk covers every block
    int rows;       // rows of an entry at most: 16, 32 or 64
    int tt, tps;    // tokens of an entry at most (rows / G), entries of a sequence and kv head
    int n_ent;      // (sequence * tps + tile) * Hkv + kv head
    int tpb;        // key tiles per block
    int ctas;       // of the attention kernel
    int ucap;       // union blocks of an entry at most
    float scale_log2;
    int *status;
    // scratch (a kernel may start while the one that writes it still runs, so it is read
    // with plain loads behind after_previous(), never as constant data: no __ldg)
    int *tiles;                 // [n_ent] key tiles of an entry (selection only)
    int *ublk;                  // [n_ent][ucap] blocks that some row of the entry selected, ascending
    unsigned long long *umask;  // [n_ent][ucap] which rows did
    int *c_open;                // [ctas] the entry that starts in the CTA's run and ends in another's, or -1
    int *c_last;                // [n_ent] the CTA in whose run the entry ends
    float *part_o;              // [ctas][2][rows][D] partial sums of exp2(s - m) v
    float2 *part_ml;            // [ctas][2][rows] their m and sum of exp2(s - m); a sum below 0: bad page
    // ---- shared prefixes: jobs that are tiles of rows with a range of keys ----
    Span *tiles_big;            // [...] 256 rows at most, for the tcgen05 kernel
    long long *off_big;         // [... + 1] key tiles before each (and kBigStart), times the kv heads
    SpanHead *head;
    int *c_first;               // [... * Hkv] the CTAs in whose runs the span on the kv head lies, to c_last
    // ---- chunks of many rows (the tcgen05 kernel): jobs of up to 256 rows ----
    bool chunk;
    int n_max;                  // blocks of a sequence at most
    int w_cap;                  // 256-row tiles of all sequences on one kv head, at most
    long long job_cap, list_cap;
    int *own_off;               // [num_seqs + 1] 256-row tiles before each sequence
    long long *unit_off;        // [w_cap + 1] key tiles before each row tile (all blocks)
    int *counts;                // [num_seqs][n_max][Hkv] rows that selected the block
    int *list_off;              // [num_seqs * n_max * Hkv], of the lists in use
    int *used_off;              // [num_seqs + 1] lists in use before each sequence: of the blocks before its last
    int2 *jobs, *halves;        // [job_cap] list, first entry: of up to 256 rows, of up to 128
    int *n_jobs;                // [3] how many of each, and how many jobs are handed out
    int *list;                  // rows of each list: (token * G + head) << 5 | slot
    int *tok;                   // [total] behind counts: a token's position + 1 (0: of no sequence, or of
                                // a refused one)
    int2 *sel;                  // [Hkv][total * G][km1] a row's past blocks, ascending, as list numbers
                                // (-1: none, kSelBad: a page outside the pool), and its place in each list
    __half *part_h;             // [Hkv][total * G][km1 + 1][D] normalised partial outputs
    float4 *part_s;             // [Hkv][total * G][km1 + 1] log2-sum-exp, scale of each 64 columns,
                                // and 1 (0: a page outside the pool)
};

struct Entry {
    int b, hk;
    int t0, nt;    // tokens [t0, t0 + nt) of the sequence's new ones
    int row0;      // packed row of token t0
    int pos0;      // position of token t0
    int state;     // kSeqOk (then nt > 0), kSeqEmpty, or kSeqBad: the first entry of a refused sequence
};

__device__ __forceinline__ Entry get_entry(const Attn &a, int e) {
    Entry x;
    x.hk = e % a.c.Hkv;
    const int t = e / a.c.Hkv;
    x.b = t / a.tps;
    x.t0 = (t - x.b * a.tps) * a.tt;
    Seq s;
    x.state = a.c.seq(x.b, s);
    x.nt = max(0, min(a.tt, s.n - x.t0));
    x.row0 = s.row0 + x.t0;
    x.pos0 = s.len - s.n + x.t0;
    if (x.state == kSeqBad ? x.t0 > 0 : x.nt == 0) x.state = kSeqEmpty;
    return x;
}

// The span that unit u lies in: the last one that starts at or before it, 128 places a
// look.  All lanes of a warp call it, with the same arguments.
__device__ __forceinline__ int span_of_unit(const long long *off, int spans, long long u, int lane) {
    int w = 0;
    for (int n = spans; n > 1;) {  // the answer is in [w, w + n)
        const int step = (n + 127) / 128;
        int last = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int at = (32 * j + lane) * step;
            last += __popc(__ballot_sync(0xffffffffu, at < n && off[w + at] <= u));
        }
        last = max(last - 1, 0);
        n = min(step, n - last * step);
        w += last * step;
    }
    return w;
}

// The rows of refused sequence s, heads [h0, h0 + nh): thread `at` of `threads`
// that clear them together.  By sequence, not by tile: its rows may be more than
// max_new, and lie where no tile begins.
__device__ __forceinline__ void clear_refused(const Attn &a, const Seq &s, int h0, int nh, int at, int threads) {
    const long long n = (long long)s.n * nh, per = a.D / 8;
    const size_t row0 = s.row0;
    for (long long i = at; i < n; i += threads) a.lse[(row0 + i / nh) * a.Hq + h0 + i % nh] = -INFINITY;
    for (long long i = at; i < n * per; i += threads)
        *reinterpret_cast<uint4 *>(a.out + ((row0 + i / per / nh) * a.Hq + h0 + i / per % nh) * a.D + i % per * 8) =
            make_uint4(0, 0, 0, 0);
    if (a.idx)
        for (long long i = at; i < n * a.topk; i += threads)
            a.idx[((row0 + i / a.topk / nh) * a.Hq + h0 + i / a.topk % nh) * a.topk + i % a.topk] = -1;
}

// the sequence of 256-row tile w (all blocks)
__device__ __forceinline__ int seq_of_tile(const Attn &a, int w) {
    int lo = 0, hi = a.c.num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.own_off[mid] <= w) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// key tiles that an entry visits
__device__ __forceinline__ int get_tiles(const Attn &a, int e) {
    if (!a.dense) return a.tiles[e];
    const Entry x = get_entry(a, e);
    return x.state == kSeqOk ? (x.pos0 + x.nt - 1) / kTile + 1 : 0;
}

// Sizes of a call whose cache has been checked (a->c is filled): MOBA_OK, or why not.
int make_attn(Attn *a, int Hq, int D, int topk);

cudaError_t launch_gate(const Attn &a, cudaStream_t st);
cudaError_t launch_chunk_gate(const Attn &a, cudaStream_t st);
// (after_gate: a kernel of this call is before it)
cudaError_t launch_rows(const Attn &a, bool after_gate, cudaStream_t st);
// chunks of many rows: row tiles, lists and jobs; then the attention and the merge
cudaError_t launch_plan(const Attn &a, bool after_gate, cudaStream_t st);
cudaError_t launch_chunk(const Attn &a, cudaStream_t st);
// shared prefixes: the big spans on the tcgen05 kernel, whose parts leave partial sums in
// slot span * Hkv + kv head + CTA (the next part has another span, head or CTA)
cudaError_t launch_chunk_spans(const Attn &a, cudaStream_t st);
// joins the partial sums of entries (row tiles of chunks) that fell into several runs
cudaError_t launch_merge_runs(const Attn &a, cudaStream_t st);

}  // namespace paged
}  // namespace moba
