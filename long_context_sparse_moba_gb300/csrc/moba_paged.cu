// moba_paged.cu -- upkeep of a paged cache: appending new tokens (with the
// pooled keys of the blocks they complete) and copying pages.
//
// Pages: "MOBA mixture of block attention for server-side long context"
// (hncyxsy.com/news/197418) section 3 (mean-pooled block keys) and section 4
// (the cache's memory); the pages describe no paged cache.
#include "moba_paged.cuh"
#include "moba_ptx.cuh"

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
// A cluster of up to eight CTAs per (block of a sequence that the new tokens touch,
// kv head): it copies the block's new tokens to their pages (16 bytes a lane) and,
// when the block is complete with them, sums the block's keys: the new ones as
// they pass through its registers, the earlier ones from the cache.  So a chunk's
// keys are read once and one launch does both.
// The block's tokens fall into 64 groups (p % 64; 128 where D is 64), eight parts of
// them, a CTA one or more parts.  A thread (column, group) takes its tokens in
// ascending order, whatever their source: a pooled key depends neither on how the
// appends were cut nor on the size of the cluster.  Sums are compensated (Kahan), as in the key pooling
// kernel; the others send theirs to the first CTA's shared memory.
// Bound: HBM for long chunks (76 us at 65536 tokens of 8 heads of 128, blocks of 512:
// the copy rate), latency for a step (2.5 us in a graph; 9 by a call, which is the host):
// the one that completes a block reads all of its keys, which eight CTAs do in two rounds
// of loads.
constexpr int kAppendThreads = 128;
constexpr int kAppendParts = 8;     // of a block's tokens; the 1, 2, 4 or 8 CTAs of a cluster take them
constexpr int kAppendPages = 512;

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
};

// the address of a shared variable's counterpart in CTA 0 of the cluster
__device__ __forceinline__ uint32_t in_first(const void *p) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(ptx::saddr(p)), "r"(0));
    return at;
}
// v to *at of CTA 0, counted by its barrier
__device__ __forceinline__ void send(uint32_t at, float v, uint32_t bar) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(at),
                 "r"(__float_as_uint(v)), "r"(bar)
                 : "memory");
}

// (s, c) += x, compensated
__device__ __forceinline__ void kahan(float &s, float &c, float x) {
    const float y = x - c, t = s + y;
    c = (t - s) - y;
    s = t;
}

// One dimension of the mean key of positions [p0, p0 + bs) of a sequence, in 64 bits,
// `first` and the later ones from the new tokens' rows (at k, dimension d of the first).
template <int D>
__device__ __noinline__ float mean64(const __nv_bfloat16 *kp, int Hkv, int psh, const int *table, int hk, int d,
                                     int p0, int bs, int first, const __nv_bfloat16 *k) {
    double sum = 0.0;
    for (int p = p0; p < p0 + bs; ++p) {
        const __nv_bfloat16 *x = p < first ? kp + ((((size_t)__ldg(table + (p >> psh)) * Hkv + hk) << psh) +
                                                   (p & ((1 << psh) - 1))) * D + d
                                           : k + (size_t)(p - first) * Hkv * D;
        sum += (double)__bfloat162float(*x);
    }
    return (float)(sum / bs);
}

template <int D, bool MAX>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendArgs a) {
    constexpr int CW = D / 8;                        // threads across a token
    constexpr int GC = kAppendThreads / CW;          // groups of a CTA
    constexpr int G = GC * kAppendParts;
    constexpr int U = 4;
    __shared__ float red[kAppendThreads][9];
    __shared__ float s_sum[kAppendParts][D], s_bad[kAppendParts];  // of CTA 0: the parts' sums
    __shared__ int s_page[kAppendPages], s_abort;
    __shared__ __align__(8) unsigned long long s_bar;
    const int rank = blockIdx.x & (a.ctas - 1), bj = (int)blockIdx.x / a.ctas, hk = blockIdx.y;
    int b, nth;  // the sequence, and which of the blocks that its new tokens touch
    Seq s;
    if (a.cand > 0) {
        b = bj / a.cand;
        nth = bj % a.cand;
    } else {
        b = a.c.tile_of(bj, 1, a.c.bs, 2, nth);
        // (no slot need lead to a sequence whose offsets are wrong)
        if (bj < a.c.num_seqs && threadIdx.x == 0 && a.c.seq(bj, s) == kSeqBad)
            atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
    }
    const int state = a.c.seq(b, s);
    if (state != kSeqOk) {
        if (state == kSeqBad && threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        return;
    }
    const int bs = a.c.bs, ps = a.c.ps;
    const int first = s.len - s.n;  // position of the first new token
    if (nth < 0 || nth > s.n / bs + 1) return;
    const int p0 = (first / bs + nth) * bs;
    if (p0 >= s.len) return;
    const bool pool = a.kbar && p0 + bs <= s.len;
    const int c1 = min(p0 + bs, s.len);
    const int t0 = pool ? p0 : max(p0, first);  // first token that is read
    if (!pool && c1 - t0 == 1 && (((t0 - p0) % G / GC) & (a.ctas - 1)) != rank)
        return;  // a step: the CTAs without the token leave
    const int col = threadIdx.x % CW;
    const int *table = a.c.table + (size_t)b * a.c.max_pages;
    const uint32_t bar = ptx::saddr(&s_bar);
    if (pool && a.ctas > 1) {
        // CTA 0's barrier stands before any CTA sends to it (all of them alike; nothing
        // is in flight yet, so the barrier costs little)
        if (rank == 0 && threadIdx.x == 0) {
            s_abort = 0;
            ptx::mbar_init(bar, 1);
            ptx::fence_mbar_init();
            ptx::mbar_expect_tx(bar, (kAppendParts - kAppendParts / a.ctas) * (D + 1) * 4);
        }
        asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
    }
    // the block's pages, looked up once (a block of more pages than the array
    // holds looks them up as it goes)
    const int g0 = t0 >> a.psh, gn = ((c1 - 1) >> a.psh) + 1 - g0;
    const bool held = gn <= kAppendPages;
    if (held) {
        for (int i = threadIdx.x; i < gn; i += kAppendThreads) s_page[i] = __ldg(table + g0 + i);
        __syncthreads();
    }
    bool bad = false;
    for (int part = rank; part < kAppendParts; part += a.ctas) {
        float acc[8], comp[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[e] = MAX ? -INFINITY : 0.f;
            comp[e] = 0.f;
        }
        for (int pb = t0 - (t0 - p0) % G + part * GC + (int)threadIdx.x / CW; pb < c1; pb += U * G) {
            uint4 x[U], y[U];
            size_t at[U];
            bool live[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int p = pb + j * G;
                live[j] = p >= t0 && p < c1;
                if (live[j]) {
                    const int page = held ? s_page[(p >> a.psh) - g0] : __ldg(table + (p >> a.psh));
                    live[j] = (unsigned)page < (unsigned)a.c.num_pages;
                    bad |= !live[j];
                    at[j] = ((((size_t)page * a.c.Hkv + hk) << a.psh) + (p & (ps - 1))) * D + col * 8;
                }
                if (live[j] && p >= first) {
                    const size_t src = ((size_t)(s.row0 + p - first) * a.c.Hkv + hk) * D + col * 8;
                    x[j] = __ldcs(reinterpret_cast<const uint4 *>(a.k + src));
                    y[j] = __ldcs(reinterpret_cast<const uint4 *>(a.v + src));
                } else if (live[j]) {
                    x[j] = *reinterpret_cast<const uint4 *>(a.kp + at[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (!live[j]) continue;
                if (pb + j * G >= first) {
                    *reinterpret_cast<uint4 *>(a.kp + at[j]) = x[j];
                    *reinterpret_cast<uint4 *>(a.vp + at[j]) = y[j];
                }
                if (pool) {
                    const __nv_bfloat162 *p2 = reinterpret_cast<const __nv_bfloat162 *>(&x[j]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float f = e & 1 ? __high2float(p2[e >> 1]) : __low2float(p2[e >> 1]);
                        if (MAX) acc[e] = fmaxf(acc[e], f);
                        else kahan(acc[e], comp[e], f);
                    }
                }
            }
        }
        if (!pool) continue;
        if (part != rank) __syncthreads();  // (the part before has been summed)
#pragma unroll
        for (int e = 0; e < 8; ++e) red[threadIdx.x][e] = acc[e];
        const bool some = __syncthreads_or(bad);
        if (threadIdx.x < D) {
            const int c8 = threadIdx.x / 8, e = threadIdx.x % 8;
            float cp = 0.f, sum = red[c8][e];
            for (int x = 1; x < GC; ++x) {
                if (MAX) sum = fmaxf(sum, red[x * CW + c8][e]);
                else kahan(sum, cp, red[x * CW + c8][e]);
            }
            // (sent and counted, no barrier: that would wait for the stores to the pages)
            if (rank == 0) s_sum[part][threadIdx.x] = sum;
            else send(in_first(&s_sum[part][threadIdx.x]), sum, in_first(&s_bar));
        }
        if (threadIdx.x == 0) {
            if (rank == 0) s_bad[part] = some ? 1.f : 0.f;
            else send(in_first(&s_bad[part]), some ? 1.f : 0.f, in_first(&s_bar));
        }
    }
    if (__syncthreads_or(bad) && threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
    if (!pool || rank != 0) return;
    if (a.ctas > 1) {
        ptx::Ctl ctl{&s_abort, a.status, kDefaultWaitLimit};
        if (!ptx::wait_bar(bar, 0, ctl)) {  // recorded as a timeout; the slot stays as it was
            ptx::drain_bar(bar, 0, kDefaultWaitLimit);
            return;
        }
    }
    if (threadIdx.x < D) {
        float sum = s_sum[0][threadIdx.x], cp = 0.f, any = s_bad[0];
#pragma unroll
        for (int r = 1; r < kAppendParts; ++r) {
            if (MAX) sum = fmaxf(sum, s_sum[r][threadIdx.x]);
            else kahan(sum, cp, s_sum[r][threadIdx.x]);
            any += s_bad[r];
        }
        if (any != 0.f) return;
        if (!MAX) sum /= (float)bs;
        // infinite keys, or a sum out of fp32's range: the compensation makes a NaN of either
        // (asking at every addition took 3 to 6 % of the call)
        if (!MAX && !(fabsf(sum) < INFINITY))
            sum = mean64<D>(a.kp, a.c.Hkv, a.psh, table, hk, threadIdx.x, p0, bs, first,
                            a.k + ((size_t)s.row0 * a.c.Hkv + hk) * D + threadIdx.x);
        const int page = __ldg(table + ((p0 + bs) >> a.psh) - 1);
        a.kbar[((size_t)page * a.c.Hkv + hk) * D + threadIdx.x] = sum;
    }
}

// ----------------------------------------------------------------------------
// page copy
// ----------------------------------------------------------------------------
// A CTA copies a part of one pair in one layer, 16 bytes a lane with several
// loads in flight.  Each CTA first looks its pair up in the whole
// destination list: a destination given twice, or a source that some pair
// overwrites, would make the result depend on the order.
// Bound: HBM; 203 us for 2500 pages of 8 x 64 x 128 (6.6 TB/s, 0.97 of the copy
// rate); 16 us for 16 pages in 8 layers, latency: 1024 CTAs of which 73 registers let 456
// in at once.  Many small pages are bound by the look at the list, n entries a CTA: 65536
// pages of 16 tokens of one head of 64 take 1.4 ms where their bytes take 84 us, 16384
// of them 137 us.
constexpr int kCopyThreads = 256;

struct CopyArgs {
    uint4 *k, *v, *kbar;  // kbar may be null
    const int *src, *dst;
    int n, num_pages, parts;
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
    const int i = blockIdx.x / a.parts, part = blockIdx.x % a.parts, l = blockIdx.y;
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
    const long long s = (long long)l * a.num_pages + src, d = (long long)l * a.num_pages + dst;
    copy_run(a.k + s * a.page16, a.k + d * a.page16, a.page16, part, a.parts);
    copy_run(a.v + s * a.page16, a.v + d * a.page16, a.page16, part, a.parts);
    if (a.kbar) copy_run(a.kbar + s * a.bar16, a.kbar + d * a.bar16, a.bar16, part, a.parts);
}

template <int D>
static cudaError_t launch_append(const AppendArgs &a, bool max, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.clusters * a.ctas), a.c.Hkv);
    cfg.blockDim = kAppendThreads;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = a.ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    note_launches(1);
    return max ? cudaLaunchKernelEx(&cfg, append_kernel<D, true>, a)
               : cudaLaunchKernelEx(&cfg, append_kernel<D, false>, a);
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
    a.psh = __builtin_ctz((unsigned)page_size);
    a.cand = (int)(((long long)a.c.max_new + block_size - 2) / block_size + 1);
    // clusters for the longest chunk of every sequence, or, where chunks are uneven
    // and that is more of them, by packed tokens (n tokens touch n / block_size + 2
    // blocks at most), which costs a search for the sequence
    a.clusters = (long long)num_seqs * a.cand;
    const long long packed = a.c.tile_slots(1, block_size, 2);
    if (packed < a.clusters) {
        a.clusters = packed;
        a.cand = 0;
    }
    if (a.clusters >= (1ll << 31) / kAppendParts) return MOBA_ERR_UNSUPPORTED;
    // CTAs to a block.  More of them shorten the step that completes one, fewer
    // leave the GPU to more blocks at once (six CTAs fit an SM).  us with 8,
    // 4, 2, 1 (D 128, 8 kv heads, blocks of 512, in a graph): a step of one sequence that
    // completes its block 4.8, 6.7, 10.4, 17.2; of 64 of which one does 9.3, 9.0, 11.1,
    // 17.9; of 256 of which three do 25.1, 18.8, 18.7, 24.1; a chunk of 65536 tokens 78,
    // 73, 75, 84, and 267, 185, 144, 117 with blocks of 64
    const double per_sm = (double)((long long)total / block_size + num_seqs) * Hkv / sm_count();
    a.ctas = per_sm * 8 <= 6 ? 8 : per_sm * 4 <= 15 ? 4 : block_size >= 512 ? 2 : 1;
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
    // (every CTA looks its pair up among all)
    if (n > 65536) return MOBA_ERR_UNSUPPORTED;
    if (Hkv > 65535 || layers > 65535 || page_size > (1 << 20) ||
        (long long)Hkv * page_size * D > (1ll << 40) / num_pages / layers)
        return MOBA_ERR_UNSUPPORTED;
    CopyArgs a;
    a.k = static_cast<uint4 *>(k_pages);
    a.v = static_cast<uint4 *>(v_pages);
    a.kbar = reinterpret_cast<uint4 *>(kbar_pages);
    a.src = src;
    a.dst = dst;
    a.n = n;
    a.num_pages = num_pages;
    a.page16 = (long long)Hkv * page_size * D / 8;
    a.bar16 = (long long)Hkv * D / 4;
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    // eight CTAs an SM (three fit at once); a part is at least 16 KB of a page
    const long long fill = (long long)sm_count() * 8;
    long long parts = (fill + (long long)n * layers - 1) / ((long long)n * layers);
    const long long most = (a.page16 + 1023) / 1024;
    if (parts > most) parts = most;
    a.parts = (int)parts;
    if ((long long)n * parts >= (1ll << 31)) return MOBA_ERR_UNSUPPORTED;
    page_copy_kernel<<<dim3((unsigned)(n * parts), layers), kCopyThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(a);
    note_launches(1);
    return cuda_result(cudaGetLastError());
}
