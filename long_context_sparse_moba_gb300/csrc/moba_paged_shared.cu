// moba_paged_shared.cu -- attention of new tokens over a paged cache whose sequences
// share long prefixes (forks of a prompt, questions on a document): a prefix is read and
// multiplied once for all the rows of its group.
//
// Pages: "MOBA mixture of block attention for server-side long context"
// (hncyxsy.com/news/197418) section 1 (long contexts served to many) and section 3
// (softmax attention over all blocks where nothing is selected).
//
// A row's softmax over prefix and own keys is that over each, joined:
//   M = max(m_i),  L = sum l_i 2^(m_i - M),  out = sum o_i 2^(m_i - M) / L
// over partial sums o_i of 2^(s - m_i) v, with their l_i, in fp32.
//   1. The plan (one CTA) checks the groups and cuts their rows into tiles of 256.
//   2. A group's rows lie one behind the other, whatever sequences they are of, so that a
//      tile with the prefix of one kv head is a job of the tcgen05 kernel of long chunks,
//      without a mask; the key tiles of all jobs are cut into equal runs, one per CTA.
//   3. What is behind the prefix is each sequence's own: few rows (a decode step) go to the
//      streaming kernel of few rows, chunks of many rows are further tiles of 2.
//   4. Every part of 2 and 3 leaves partial sums, which the merge joins, a warp a row.
#include "moba_paged_attn.cuh"
#include "moba_mma.cuh"

namespace moba {
namespace paged {
namespace {

constexpr int kMergeWarps = 8;

// Partial sums of a row joined so far: maximum (log2) and sum, and the lane's columns.
template <int V>
struct Joined {
    float M = -INFINITY, L = 0.f, acc[V] = {};
    bool bad = false;

    // parts of slots p0, p0 + step, ..., n of them, each row of D values
    __device__ __forceinline__ void add(const float *o, const float2 *ml, size_t p0, size_t step, int n, int lane) {
        constexpr int U = 4, D = 32 * V;
        for (int i = 0; i < n; i += U) {
            float2 s[U];
            float v[U][V];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                s[j] = make_float2(-INFINITY, 0.f);
                if (i + j < n) {
                    const size_t p = p0 + (size_t)(i + j) * step;
                    s[j] = ml[p];
#pragma unroll
                    for (int k = 0; k < V; k += 2)
                        *reinterpret_cast<float2 *>(&v[j][k]) =
                            *reinterpret_cast<const float2 *>(o + p * D + lane * V + k);
                }
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                bad |= s[j].y < 0.f;
                if (s[j].y == 0.f) continue;  // no part, or one without a key for this row
                const float mn = fmaxf(M, s[j].x), ref = mn == -INFINITY ? 0.f : mn;
                const float f = mma::fast_exp2(M - ref), g = mma::fast_exp2(s[j].x - ref);
                M = mn;
                L = fmaf(s[j].y, g, L * f);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] = fmaf(v[j][k], g, acc[k] * f);
            }
        }
    }
};

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) merge_shared_kernel(Attn a) {
    constexpr int V = D / 32;
    after_previous();
    const int lane = threadIdx.x & 31, G = a.G, Hkv = a.c.Hkv;
    const long long row = (long long)blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= (long long)a.c.total * a.Hq) return;
    const int t = (int)(row / a.Hq), h = (int)(row - (long long)t * a.Hq), hk = h / G, gh = h - hk * G;
    const int b = a.c.seq_of_row(t, lane);
    Seq s;
    if (a.c.seq(b, s) != kSeqOk || t < s.row0 || t >= s.row0 + s.n) return;
    const int j = t - s.row0;
    const int pre = a.pre_off[a.n_groups], tiles = pre + (a.chunk ? a.own_off[a.c.num_seqs] : 0);
    const long long total = a.unit_off[tiles], runs = total < a.ctas ? total : a.ctas;
    Joined<V> x;
    // the parts of a tile's row: those of the CTAs whose runs [total c / runs, total (c + 1) /
    // runs) its key tiles on this kv head lie in
    auto tile = [&](int r) {
        const int w = r / kJobRows;
        const long long u0 = a.unit_off[w], T = (a.unit_off[w + 1] - u0) / Hkv, u = u0 + hk * T;
        const int c0 = (int)(((u + 1) * runs - 1) / total), c1 = (int)(((u + T) * runs - 1) / total);
        const size_t slot = (size_t)w * Hkv + hk + c0;
        x.add(a.part_o, a.part_ml, slot * kJobRows + r % kJobRows, kJobRows, c1 - c0 + 1, lane);
    };
    if (a.first[b] > 0) tile(a.pre_row[b] + j * G + gh);
    if (a.chunk) {
        // (rows without a tile: from offsets that overlap)
        const int r = j * G + gh;
        if (a.own_off[b] + r / kJobRows >= a.own_off[b + 1]) return;
        tile((pre + a.own_off[b]) * kJobRows + r);
    } else {
        const int e = (b * a.tps + j / a.tt) * Hkv + hk;
        const int c0 = max(a.c_first[e], 0), c1 = min(a.c_last[e], a.ctas - 1);
        x.add(a.own_o, a.own_ml, (size_t)(e + c0) * a.rows + j % a.tt * G + gh, a.rows, c1 - c0 + 1, lane);
    }
    const float inv = 1.f / x.L;
#pragma unroll
    for (int k = 0; k < V; k += 2)
        *reinterpret_cast<uint32_t *>(a.out + (size_t)row * D + lane * V + k) =
            x.bad ? 0u : mma::pack_bf16(x.acc[k] * inv, x.acc[k + 1] * inv);
    if (lane == 0) a.lse[row] = x.bad ? -INFINITY : (x.M + log2f(x.L)) * 0.69314718055994530942f;
}

size_t scratch(Attn *a, void *base) {
    size_t off = 0;
    auto take = [&](size_t bytes) -> void * {
        void *p = base ? static_cast<char *>(base) + off : nullptr;
        off = (off + bytes + 255) & ~size_t(255);
        return p;
    };
    const size_t ns = a->c.num_seqs, ng = a->n_groups, tiles = (size_t)a->pre_cap + (a->chunk ? a->w_cap : 0);
    a->first = static_cast<int *>(take(4 * ns));
    a->pre_row = static_cast<int *>(take(4 * ns));
    a->rep = static_cast<int *>(take(4 * (ng + 1)));
    a->pre_off = static_cast<int *>(take(4 * (ng + 1)));
    a->unit_off = static_cast<long long *>(take(8 * (tiles + 1)));
    const size_t parts = tiles ? (tiles * a->c.Hkv + a->ctas) * kJobRows : 0;
    a->part_ml = static_cast<float2 *>(take(sizeof(float2) * parts));
    a->part_o = static_cast<float *>(take(sizeof(float) * parts * a->D));
    if (a->chunk) {
        a->own_off = static_cast<int *>(take(4 * (ns + 1)));
    } else {
        const size_t own = ((size_t)a->n_ent + a->ctas) * a->rows;
        a->c_first = static_cast<int *>(take(4 * (size_t)a->n_ent));
        a->c_last = static_cast<int *>(take(4 * (size_t)a->n_ent));
        a->own_ml = static_cast<float2 *>(take(sizeof(float2) * own));
        a->own_o = static_cast<float *>(take(sizeof(float) * own * a->D));
    }
    return off;
}

// Sizes of a call whose cache has been checked.
int make_shared(Attn *a, int Hq, int D, int n_groups) {
    if (n_groups < 0) return MOBA_ERR_INVALID_ARG;
    if (n_groups > 65535) return MOBA_ERR_UNSUPPORTED;
    const int rc = make_attn(a, Hq, D, 1 << 30);
    if (rc != MOBA_OK) return rc;
    a->shared = true;
    a->n_groups = n_groups;
    const long long rows = (long long)a->c.total * a->G;
    if (rows >= (1ll << 26)) return MOBA_ERR_UNSUPPORTED;
    // a tile that is not full for every group with rows
    long long some = n_groups < a->c.num_seqs ? n_groups : a->c.num_seqs;
    if (some > a->c.total) some = a->c.total;
    a->pre_cap = n_groups ? (int)(rows / kJobRows + some) : 0;
    const long long tiles = a->pre_cap + (a->chunk ? (long long)a->w_cap : 0);
    if (tiles * a->c.Hkv >= (1ll << 30) || a->n_ent >= (1 << 30)) return MOBA_ERR_UNSUPPORTED;
    return MOBA_OK;
}

template <int D>
cudaError_t launch_merge(const Attn &a, cudaStream_t st) {
    const long long rows = (long long)a.c.total * a.Hq;
    note_launches(1);
    return launch_after(merge_shared_kernel<D>, dim3((unsigned)((rows + kMergeWarps - 1) / kMergeWarps)),
                        dim3(32 * kMergeWarps), 0, st, a);
}

}  // namespace
}  // namespace paged
}  // namespace moba

using namespace moba;
using namespace moba::paged;

// (no block is ever selected: any block size does for the cache's checks)
static int any_block(int page_size) { return page_size < 64 ? 64 : page_size; }

MOBA_EXPORT size_t moba_paged_attn_shared_workspace_size(int num_seqs, int n_groups, int total, int max_new, int Hq,
                                                         int Hkv, int D, int page_size, int max_pages) {
    Attn a = {};
    // any non-null, aligned addresses: only the sizes matter here
    const void *some = reinterpret_cast<const void *>(256);
    const int32_t *ints = static_cast<const int32_t *>(some);
    if (make_cache(&a.c, some, some, nullptr, ints, ints, ints, num_seqs, total, max_new, Hkv, D, 1, page_size,
                   max_pages, any_block(page_size)) != MOBA_OK ||
        make_shared(&a, Hq, D, n_groups) != MOBA_OK)
        return 0;
    return scratch(&a, nullptr);
}

MOBA_EXPORT int moba_paged_attn_shared(const void *q, const void *k_pages, const void *v_pages,
                                       const int32_t *page_table, const int32_t *cu_new, const int32_t *cache_lens,
                                       const int32_t *cu_groups, const int32_t *prefix_lens, void *out, float *lse,
                                       int num_seqs, int n_groups, int total, int max_new, int Hq, int Hkv, int D,
                                       int num_pages, int page_size, int max_pages, void *workspace,
                                       size_t workspace_bytes, void *stream) {
    if (!q || !out || !lse || (n_groups > 0 && (!cu_groups || !prefix_lens))) return MOBA_ERR_INVALID_ARG;
    Attn a = {};
    int rc = make_cache(&a.c, k_pages, v_pages, nullptr, page_table, cu_new, cache_lens, num_seqs, total, max_new,
                        Hkv, D, num_pages, page_size, max_pages, any_block(page_size));
    if (rc == MOBA_OK) rc = make_shared(&a, Hq, D, n_groups);
    if (rc != MOBA_OK) return rc;
    if (misaligned16(q) || misaligned16(out) ||
        ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(cu_groups) |
          reinterpret_cast<uintptr_t>(prefix_lens)) & 3))
        return MOBA_ERR_INVALID_ARG;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k_pages);
    a.v = static_cast<const __nv_bfloat16 *>(v_pages);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.cu_groups = cu_groups;
    a.prefix_lens = prefix_lens;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t need = scratch(&a, nullptr);
    if (workspace && (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return MOBA_ERR_WORKSPACE;
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    void *own = nullptr;
    if (!workspace) {
        const cudaError_t e = cudaMallocAsync(&own, need, st);
        if (e != cudaSuccess) return cuda_result(e);
        workspace = own;
    }
    scratch(&a, workspace);
    cudaError_t e = launch_plan_shared(a, st);
    if (e == cudaSuccess && (a.n_groups || a.chunk)) e = launch_chunk_shared(a, st);
    if (e == cudaSuccess && !a.chunk) e = launch_rows(a, true, st);
    if (e == cudaSuccess) e = D == 64 ? launch_merge<64>(a, st) : launch_merge<128>(a, st);
    if (own) {
        const cudaError_t f = cudaFreeAsync(own, st);
        if (e == cudaSuccess) e = f;
    }
    return cuda_result(e);
}
