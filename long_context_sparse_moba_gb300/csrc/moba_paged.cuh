// moba_paged.cuh -- the paged cache as its kernels see it.
#pragma once

#include <atomic>

#include "moba.h"
#include "moba_internal.cuh"

namespace moba {
namespace paged {

// The new tokens of one sequence.
struct Seq {
    int row0;  // its first row of the packed tensors
    int n;     // new tokens
    int len;   // tokens in the cache, with the new ones
};
enum { kSeqOk = 0, kSeqEmpty = 1, kSeqBad = 2 };

struct Cache {
    const int *table;  // [num_seqs][max_pages]
    const int *cu;     // [num_seqs + 1]
    const int *lens;   // [num_seqs]
    int num_seqs, total, max_new, Hkv, num_pages, ps, max_pages, bs;

    // Reads and checks sequence b's offsets and length.  kSeqBad: its rows, if
    // any, are [s.row0, s.row0 + s.n) after clamping into [0, total), which may be
    // more than max_new, and nothing else of it may be used.
    __device__ __forceinline__ int seq(int b, Seq &s) const {
        return check(__ldg(cu + b), __ldg(cu + b + 1), __ldg(lens + b), s);
    }
    // (the same by plain loads: see launch_after)
    __device__ __forceinline__ int seq_now(int b, Seq &s) const { return check(cu[b], cu[b + 1], lens[b], s); }
    __device__ __forceinline__ int check(int lo, int hi, int len, Seq &s) const {
        s.row0 = lo;
        s.len = len;
        const bool rows_ok = lo >= 0 && hi >= lo && hi <= total && hi - lo <= max_new;
        if (rows_ok) {
            s.n = hi - lo;
            if (s.n <= s.len && (long long)s.len <= (long long)max_pages * ps)
                return s.n > 0 ? kSeqOk : kSeqEmpty;
            return kSeqBad;
        }
        s.row0 = min(max(lo, 0), total);
        s.n = min(max(hi, s.row0), total) - s.row0;
        return kSeqBad;
    }

    // The sequence that may hold packed row t: the last one that starts at or before it, 32
    // places a look, by plain loads.  All lanes of a warp call it, with the same t.
    __device__ __forceinline__ int seq_of_row(int t, int lane) const {
        int lo = 0, n = num_seqs;  // the answer is in [lo, lo + n)
        while (n > 1) {
            const int step = (n + 31) / 32;
            const bool below = lane * step < n && cu[lo + lane * step] <= t;
            const unsigned some = __ballot_sync(0xffffffffu, below);
            const int last = some ? 31 - __clz(some) : 0;
            n = min(step, n - last * step);
            lo += last * step;
        }
        return lo;
    }

    // Tiles of `rows` rows (head rows of a group of G, numbered token * G + head)
    // without a table: sequence b's begin at slot cu[b] * G / rows + spare * b,
    // which leaves room for `spare` tiles of every sequence that are not full.
    // There are tile_slots of them; a slot's sequence, and its tile (any number: it
    // may lie behind the sequence's end).
    __device__ __forceinline__ int tile_of(int slot, int G, int rows, int spare, int &tile) const {
        return tile_by([](const int *p) { return __ldg(p); }, slot, G, rows, spare, tile);
    }
    template <typename Read>
    __device__ __forceinline__ int tile_by(Read read, int slot, int G, int rows, int spare, int &tile) const {
        int lo = 0, hi = num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)read(cu + mid) * G / rows + (long long)spare * mid <= slot) lo = mid; else hi = mid - 1;
        }
        tile = (int)(slot - ((long long)read(cu + lo) * G / rows + (long long)spare * lo));
        return lo;
    }
    __host__ __device__ long long tile_slots(int G, int rows, int spare) const {
        return (long long)total * G / rows + (long long)spare * num_seqs;
    }
};

// A kernel that follows another one of the same call: its CTAs may start while
// that one drains, and each begins with after_previous(), which waits for all of
// its results (or ends with it, where it needs none of them).  Every CTA of every kernel
// in such a row has to make that wait, so that a kernel's end implies the end of all before it.
// (The first kernel of some calls is launched so too: what is before it on the stream has then
// ended when its wait has; 2 us less from call to call.  What wrote its operands may run while it
// is there already, so they are no constant data to it: behind the wait, and by plain loads, which
// stay behind it.  It lets the next kernel in behind its wait: to that one they are constant.)
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}
__device__ __forceinline__ void after_previous() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
// the next kernel's CTAs may be brought in as this one's leave
__device__ __forceinline__ void let_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The dynamic shared memory limit of kernel K, raised once per device.
template <auto K>
cudaError_t allow_smem(int bytes) {
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t rc = cudaGetDevice(&dev);
    if (rc != cudaSuccess) return rc;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    rc = cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (rc == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return rc;
}

// Appending (moba_paged.cu), or pooling what has been appended.
struct AppendArgs {
    Cache c;
    const __nv_bfloat16 *k, *v;  // [total][Hkv][D]
    __nv_bfloat16 *kp, *vp;
    float *kbar;
    int cand;  // blocks that a sequence's new tokens touch, at most; 0: clusters by packed tokens
    int psh;   // log2(page size)
    long long clusters;
    int ctas;  // of a cluster
    int *status;
    unsigned long long *ready, token;  // pooling alone: where the kernel before it leaves the call's token
};
// Pooling alone, behind a kernel of the same call that writes the pages and, behind its own wait
// and before it lets this one in, releases the token: its arguments (MOBA_OK, or why not), and
// the launch.
int make_pool(AppendArgs *a, const Cache &c, void *k_pages, float *kbar_pages, int *status);
cudaError_t launch_pool(const AppendArgs &a, int D, bool max, cudaStream_t st);

// Host checks shared by the entry points; fills c.
int make_cache(Cache *c, const void *k_pages, const void *v_pages, const float *kbar_pages,
               const int32_t *table, const int32_t *cu, const int32_t *lens, int num_seqs,
               int total, int max_new, int Hkv, int D, int num_pages, int page_size, int max_pages,
               int block_size);

}  // namespace paged
}  // namespace moba
