// moba_paged.cu -- upkeep of a paged cache: appending new tokens (with the
// pooled keys of the blocks they complete) and copying pages.
//
// Pages: "MOBA mixture of block attention for server-side long context"
// (hncyxsy.com/news/197418) section 3 (mean-pooled block keys) and section 4
// (the cache's memory); the pages describe no paged cache.
#include "moba_paged.cuh"

namespace moba {
namespace paged {

int make_cache(Cache *c, const void *k_pages, const void *v_pages, const float *kbar_pages,
               const int32_t *table, const int32_t *cu, const int32_t *lens, int num_seqs,
               int total, int max_new, int Hkv, int D, int num_pages, int page_size, int max_pages,
               int block_size) {
    if (!k_pages || !v_pages || !table || !cu || !lens) return MOBA_ERR_INVALID_ARG;
    if (num_seqs < 1 || total < 1 || max_new < 1 || Hkv < 1 || num_pages < 1 || max_pages < 1)
        return MOBA_ERR_INVALID_ARG;
    if (page_size < 16 || (page_size & (page_size - 1))) return MOBA_ERR_INVALID_ARG;
    if (block_size < 64 || block_size % 64 || block_size % page_size) return MOBA_ERR_INVALID_ARG;
    if (misaligned16(k_pages) || misaligned16(v_pages) || misaligned16(kbar_pages))
        return MOBA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(cu) |
         reinterpret_cast<uintptr_t>(lens)) & 3)
        return MOBA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return MOBA_ERR_UNSUPPORTED;
    if (total >= kMaxTokens || num_seqs > 65535 || Hkv > 65535) return MOBA_ERR_UNSUPPORTED;
    // positions, and rows of a pool ([page][head][token]), are 32-bit
    if ((long long)max_pages * page_size >= (1ll << 30)) return MOBA_ERR_UNSUPPORTED;
    if ((long long)Hkv * page_size > ((1ll << 31) - 1) / num_pages) return MOBA_ERR_UNSUPPORTED;
    if (max_new > total) max_new = total;
    c->table = table;
    c->cu = cu;
    c->lens = lens;
    c->num_seqs = num_seqs;
    c->total = total;
    c->max_new = max_new;
    c->Hkv = Hkv;
    c->num_pages = num_pages;
    c->ps = page_size;
    c->max_pages = max_pages;
    c->bs = block_size;
    return MOBA_OK;
}

// ----------------------------------------------------------------------------
// append
// ----------------------------------------------------------------------------
// One CTA per (block of a sequence that the new tokens touch, kv head, k or v):
// it copies the block's new tokens to their pages (16 bytes a lane) and, for k,
// when the block is complete with them, sums the block's keys: the new ones as
// they pass through its registers, the earlier ones from the cache.  So a
// chunk's keys are read once and one launch does both.
// Thread (column c, group g) takes the tokens with p % G == g of the block,
// ascending, whatever their source: a pooled key does not depend on how the
// appends were cut.  Sums are compensated (Kahan), as in the key pooling
// kernel.  Bound: HBM.
constexpr int kAppendThreads = 256;

struct AppendArgs {
    Cache c;
    const __nv_bfloat16 *k, *v;  // [total][Hkv][D]
    __nv_bfloat16 *kp, *vp;
    float *kbar;
    int cand;  // blocks that a sequence's new tokens touch, at most
    int *status;
};

template <int D, bool MAX>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
    constexpr int CW = D / 8;                     // threads across a token
    constexpr int G = kAppendThreads / CW;        // tokens in flight
    __shared__ float red[kAppendThreads][9];
    const int b = blockIdx.x / a.cand, hk = blockIdx.y;
    const bool is_k = blockIdx.z == 0;
    Seq s;
    const int state = a.c.seq(b, s);
    if (state != kSeqOk) {
        if (state == kSeqBad && threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        return;
    }
    const int bs = a.c.bs, ps = a.c.ps;
    const int first = s.len - s.n;  // position of the first new token
    const int p0 = (first / bs + (int)(blockIdx.x % a.cand)) * bs;
    if (p0 >= s.len) return;
    const bool pool = is_k && a.kbar && p0 + bs <= s.len;
    const int col = threadIdx.x % CW, g = threadIdx.x / CW;
    const int c1 = min(p0 + bs, s.len);
    const int t0 = pool ? p0 : max(p0, first);  // first token that is read
    const __nv_bfloat16 *src = is_k ? a.k : a.v;
    __nv_bfloat16 *pages = is_k ? a.kp : a.vp;
    const int *table = a.c.table + (size_t)b * a.c.max_pages;
    float acc[8], comp[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        acc[e] = MAX ? -INFINITY : 0.f;
        comp[e] = 0.f;
    }
    bool bad = false;
    constexpr int U = 8;
    for (int pb = t0 - (t0 - p0) % G + g; pb < c1; pb += U * G) {
        uint4 x[U];
        __nv_bfloat16 *dst[U];
        bool live[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int p = pb + j * G;
            live[j] = p >= t0 && p < c1;
            if (live[j]) {
                const int page = __ldg(table + p / ps);
                live[j] = (unsigned)page < (unsigned)a.c.num_pages;
                bad |= !live[j];
                dst[j] = pages + (((size_t)page * a.c.Hkv + hk) * ps + p % ps) * D + col * 8;
            }
            if (live[j])
                x[j] = p >= first
                           ? __ldcs(reinterpret_cast<const uint4 *>(
                                 src + ((size_t)(s.row0 + p - first) * a.c.Hkv + hk) * D + col * 8))
                           : *reinterpret_cast<const uint4 *>(dst[j]);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (!live[j]) continue;
            if (pb + j * G >= first) *reinterpret_cast<uint4 *>(dst[j]) = x[j];
            if (pool) {
                const __nv_bfloat162 *p2 = reinterpret_cast<const __nv_bfloat162 *>(&x[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float f = e & 1 ? __high2float(p2[e >> 1]) : __low2float(p2[e >> 1]);
                    if (MAX) {
                        acc[e] = fmaxf(acc[e], f);
                    } else {
                        const float y = f - comp[e];
                        const float t = acc[e] + y;
                        comp[e] = (t - acc[e]) - y;
                        acc[e] = t;
                    }
                }
            }
        }
    }
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
    if (!pool || bad) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) red[threadIdx.x][e] = acc[e];
    __syncthreads();
    if (threadIdx.x < D) {
        const int c8 = threadIdx.x / 8, e = threadIdx.x % 8;
        float sum = red[c8][e];
        if (MAX) {
            for (int x = 1; x < G; ++x) sum = fmaxf(sum, red[x * CW + c8][e]);
        } else {
            float cp = 0.f;
            for (int x = 1; x < G; ++x) {
                const float y = red[x * CW + c8][e] - cp;
                const float t = sum + y;
                cp = (t - sum) - y;
                sum = t;
            }
            sum /= (float)bs;
        }
        const int page = __ldg(table + (p0 + bs) / ps - 1);
        a.kbar[((size_t)page * a.c.Hkv + hk) * D + threadIdx.x] = sum;
    }
}

// ----------------------------------------------------------------------------
// page copy
// ----------------------------------------------------------------------------
// CTA (i, part) copies its part of pair i in every layer, 16 bytes a lane with
// several loads in flight.  Each CTA first looks its pair up in the whole
// destination list: a destination given twice, or a source that some pair
// overwrites, would make the result depend on the order.
constexpr int kCopyThreads = 256;

struct CopyArgs {
    uint4 *k, *v, *kbar;  // kbar may be null
    const int *src, *dst;
    int n, layers, num_pages, parts;
    long long page16, bar16;  // 16-byte units of a page of k (or v), of a pooled key slot
    int *status;
};

__device__ __forceinline__ void copy_run(const uint4 *__restrict__ s, uint4 *__restrict__ d,
                                         long long n, int part, int parts) {
    const long long per = (n + parts - 1) / parts;
    const long long lo = per * part, hi = min(lo + per, n);
    constexpr int U = 8;
    for (long long i = lo + threadIdx.x; i < hi; i += U * kCopyThreads) {
        uint4 x[U];
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i + j * kCopyThreads < hi) x[j] = __ldcs(s + i + j * kCopyThreads);
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (i + j * kCopyThreads < hi) __stcs(d + i + j * kCopyThreads, x[j]);
    }
}

__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(CopyArgs a) {
    const int i = blockIdx.x / a.parts, part = blockIdx.x % a.parts;
    const int src = __ldg(a.src + i), dst = __ldg(a.dst + i);
    bool bad = (unsigned)src >= (unsigned)a.num_pages || (unsigned)dst >= (unsigned)a.num_pages;
    for (int j = threadIdx.x; j < a.n; j += kCopyThreads) {
        const int d = __ldg(a.dst + j);
        bad |= d == src || (d == dst && j != i);
    }
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        return;
    }
    for (int l = 0; l < a.layers; ++l) {
        const long long s = (long long)l * a.num_pages + src, d = (long long)l * a.num_pages + dst;
        copy_run(a.k + s * a.page16, a.k + d * a.page16, a.page16, part, a.parts);
        copy_run(a.v + s * a.page16, a.v + d * a.page16, a.page16, part, a.parts);
        if (a.kbar) copy_run(a.kbar + s * a.bar16, a.kbar + d * a.bar16, a.bar16, part, a.parts);
    }
}

template <int D>
static cudaError_t launch_append(const AppendArgs &a, bool max, cudaStream_t st) {
    const dim3 grid(a.c.num_seqs * a.cand, a.c.Hkv, 2);
    if (max) append_kernel<D, true><<<grid, kAppendThreads, 0, st>>>(a);
    else append_kernel<D, false><<<grid, kAppendThreads, 0, st>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

}  // namespace paged
}  // namespace moba

using namespace moba;
using namespace moba::paged;

MOBA_EXPORT int moba_paged_append(const void *k, const void *v, void *k_pages, void *v_pages,
                                  float *kbar_pages, const int32_t *page_table,
                                  const int32_t *cu_new, const int32_t *cache_lens, int num_seqs,
                                  int total, int max_new, int Hkv, int D, int num_pages,
                                  int page_size, int max_pages, int block_size,
                                  const moba_options_t *options, void *stream) {
    if (!k || !v) return MOBA_ERR_INVALID_ARG;
    int pool = MOBA_POOL_MEAN;
    if (options) {
        if (options->pooling != MOBA_POOL_MEAN && options->pooling != MOBA_POOL_MAX)
            return MOBA_ERR_INVALID_ARG;
        pool = options->pooling;
    }
    AppendArgs a;
    const int rc = make_cache(&a.c, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens,
                              num_seqs, total, max_new, Hkv, D, num_pages, page_size, max_pages,
                              block_size);
    if (rc != MOBA_OK) return rc;
    if (misaligned16(k) || misaligned16(v)) return MOBA_ERR_INVALID_ARG;
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.kp = static_cast<__nv_bfloat16 *>(k_pages);
    a.vp = static_cast<__nv_bfloat16 *>(v_pages);
    a.kbar = kbar_pages;
    a.cand = (int)(((long long)a.c.max_new + block_size - 2) / block_size + 1);
    if ((long long)num_seqs * a.cand >= (1ll << 31)) return MOBA_ERR_UNSUPPORTED;
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool max = pool == MOBA_POOL_MAX;
    return cuda_result(D == 64 ? launch_append<64>(a, max, st) : launch_append<128>(a, max, st));
}

MOBA_EXPORT int moba_page_copy(void *k_pages, void *v_pages, float *kbar_pages, const int32_t *src,
                               const int32_t *dst, int n, int layers, int num_pages, int Hkv,
                               int D, int page_size, void *stream) {
    if (!k_pages || !v_pages || !src || !dst || n < 1 || layers < 1 || num_pages < 1 || Hkv < 1)
        return MOBA_ERR_INVALID_ARG;
    if (page_size < 16 || (page_size & (page_size - 1))) return MOBA_ERR_INVALID_ARG;
    if (misaligned16(k_pages) || misaligned16(v_pages) || misaligned16(kbar_pages))
        return MOBA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & 3)
        return MOBA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return MOBA_ERR_UNSUPPORTED;
    if (Hkv > 65535 || page_size > (1 << 20) ||
        (long long)Hkv * page_size * D > (1ll << 40) / num_pages / layers)
        return MOBA_ERR_UNSUPPORTED;
    CopyArgs a;
    a.k = static_cast<uint4 *>(k_pages);
    a.v = static_cast<uint4 *>(v_pages);
    a.kbar = reinterpret_cast<uint4 *>(kbar_pages);
    a.src = src;
    a.dst = dst;
    a.n = n;
    a.layers = layers;
    a.num_pages = num_pages;
    a.page16 = (long long)Hkv * page_size * D / 8;
    a.bar16 = (long long)Hkv * D / 4;
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    // enough CTAs to fill the GPU; a part is at least 16 KB of a page
    const long long fill = (long long)sm_count() * 8;
    long long parts = (fill + n - 1) / n;
    const long long most = (a.page16 + 1023) / 1024;
    if (parts > most) parts = most;
    a.parts = (int)parts;
    if ((long long)n * parts >= (1ll << 31)) return MOBA_ERR_UNSUPPORTED;
    page_copy_kernel<<<(unsigned)(n * parts), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
    note_launches(1);
    return cuda_result(cudaGetLastError());
}
