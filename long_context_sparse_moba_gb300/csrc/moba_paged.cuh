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
        const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
        s.row0 = lo;
        s.len = __ldg(lens + b);
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

    // Tiles of `rows` rows (head rows of a group of G, numbered token * G + head)
    // without a table: sequence b's begin at slot cu[b] * G / rows + spare * b,
    // which leaves room for `spare` tiles of every sequence that are not full.
    // There are tile_slots of them; a slot's sequence, and its tile (any number: it
    // may lie behind the sequence's end).
    __device__ __forceinline__ int tile_of(int slot, int G, int rows, int spare, int &tile) const {
        int lo = 0, hi = num_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if ((long long)__ldg(cu + mid) * G / rows + (long long)spare * mid <= slot) lo = mid; else hi = mid - 1;
        }
        tile = (int)(slot - ((long long)__ldg(cu + lo) * G / rows + (long long)spare * lo));
        return lo;
    }
    __host__ __device__ long long tile_slots(int G, int rows, int spare) const {
        return (long long)total * G / rows + (long long)spare * num_seqs;
    }
};

// A kernel that follows another one of the same call: its CTAs may start while
// that one drains, and each begins with after_previous(), which waits for all of
// its results.  Every CTA of every kernel in such a row has to make that wait, so
// that a kernel's end implies the end of all before it.
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

// Host checks shared by the entry points; fills c.
int make_cache(Cache *c, const void *k_pages, const void *v_pages, const float *kbar_pages,
               const int32_t *table, const int32_t *cu, const int32_t *lens, int num_seqs,
               int total, int max_new, int Hkv, int D, int num_pages, int page_size, int max_pages,
               int block_size);

}  // namespace paged
}  // namespace moba
