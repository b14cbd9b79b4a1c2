// moba_paged.cuh -- the paged cache as its kernels see it.
#pragma once

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
    // any, are [s.row0, s.row0 + s.n) after clamping into [0, total) and to
    // max_new rows, and nothing else of it may be used.
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
        const int end = min(max(hi, s.row0), total);
        s.n = min(end - s.row0, max_new);
        return kSeqBad;
    }
};

// Host checks shared by the entry points; fills c.
int make_cache(Cache *c, const void *k_pages, const void *v_pages, const float *kbar_pages,
               const int32_t *table, const int32_t *cu, const int32_t *lens, int num_seqs,
               int total, int max_new, int Hkv, int D, int num_pages, int page_size, int max_pages,
               int block_size);

}  // namespace paged
}  // namespace moba
