// moba_paged_rows.cu -- attention of a few query rows (up to 64 that share a kv
// head: the heads of a decode step, or of a few new tokens) over a paged cache.
//
// Pages: "When a MoBA reproduction will not run" (mhpq.cn/news/582794) section
// 3.3 (softmax attention over the selected blocks) and "MOBA mixture of block
// attention for server-side long context" (hncyxsy.com/news/197418) section 3.
//
// An entry's rows attend to the keys of the blocks that any of them selected
// (or of all blocks), 64 keys a tile, each row masked to its own blocks and to
// its own position.  Bound: HBM, so every key tile is read once for all rows of
// its kv head.  All tiles of all entries form one sequence that is cut into
// equal runs, one per CTA, whatever the sequences' lengths; an entry that falls
// into several runs leaves partial sums (at most two per CTA) that the merge
// kernel joins.
// Four warps: 16 * RW rows, 4 / RW warps side by side on a tile's keys, joined
// through shared memory at the end of an entry.  Scores and outputs on
// mma.sync; one pass with running maximum and sum in 32 bits; P is rounded to
// bf16 for the second product, as the prefill kernels do.
#include "moba_mma.cuh"
#include "moba_paged_attn.cuh"

namespace moba {
namespace paged {
namespace {

using namespace mma;

constexpr int kThreads = 128;
constexpr int kStages = 5;

template <int D>
struct RowsSmem {
    static constexpr uint32_t kTileBytes = kTile * D * 2;         // K or V
    static constexpr uint32_t kComb = kStages * 2 * kTileBytes;   // [64][D] fp32
    static constexpr uint32_t kBytes = kComb + kMaxRows * D * 4;
};

// Where a run stands: tile i of entry e's T tiles.
struct Cursor {
    int e, i, T;
    __device__ __forceinline__ void next(const Attn &a) {
        if (++i < T) return;
        i = 0;
        do {
            ++e;
        } while (e < a.n_ent && (T = get_tiles(a, e)) == 0);
    }
};

template <int D, int RW>
__global__ void __launch_bounds__(kThreads, 1) rows_kernel(Attn a) {
    using S = RowsSmem<D>;
    constexpr int KS = D / 16;
    constexpr int KW = 4 / RW;         // warps along the keys
    constexpr int KPW = kTile / KW;    // keys of a tile per warp
    constexpr int ROWS = 16 * RW;
    constexpr int CH = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_warp[4], s_base;
    __shared__ int s_e0, s_bad[kStages];
    __shared__ float s_m[kMaxRows], s_l[kMaxRows];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    const uint32_t s0 = smem_u32(smem);
    float *comb = reinterpret_cast<float *>(smem + S::kComb);

    // ---- this CTA's run of the tiles of all entries ----
    const int per = (a.n_ent + kThreads - 1) / kThreads;
    const int lo = min(tid * per, a.n_ent), hi = min(lo + per, a.n_ent);
    long long sum = 0;
    for (int e = lo; e < hi; ++e) sum += get_tiles(a, e);
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    if (tid < kStages) s_bad[tid] = 0;
    __syncthreads();
    long long before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    // at least one tile each, so that an entry's runs are those of adjacent CTAs
    const long long runs = total < (long long)gridDim.x ? total : (long long)gridDim.x;
    if (cta >= runs) return;
    const long long u0 = total * cta / runs, u1 = total * (cta + 1) / runs;
    if (u0 >= before && u0 < before + sum) {
        int e = lo;
        long long p = before;
        for (int t; u0 >= p + (t = get_tiles(a, e)); ++e) p += t;
        s_e0 = e;
        s_base = p;
    }
    __syncthreads();
    Cursor cur{s_e0, (int)(u0 - s_base), get_tiles(a, s_e0)};
    Cursor ld = cur;
    const int n = (int)(u1 - u0);

    // first key and row mask of a tile
    auto tile_of = [&](const Cursor &c, unsigned long long &mask) -> int {
        if (a.dense) {
            mask = ~0ull;
            return c.i * kTile;
        }
        const int u = c.i / a.tpb;
        mask = a.umask[(size_t)c.e * a.ucap + u];
        return a.ublk[(size_t)c.e * a.ucap + u] * a.c.bs + (c.i - u * a.tpb) * kTile;
    };
    // copies of tile j of the run into its stage: keys behind the entry's last
    // row are zeros, so that nothing unwritten meets the products
    auto load = [&](int j) {
        if (j < n) {
            const Entry x = get_entry(a, ld.e);
            unsigned long long mask;
            const int key0 = tile_of(ld, mask), end = x.pos0 + x.nt;
            const int *table = a.c.table + (size_t)x.b * a.c.max_pages;
            const int st = j % kStages;
            const uint32_t dk = s0 + st * 2 * S::kTileBytes, dv = dk + S::kTileBytes;
#pragma unroll
            for (int it = 0; it < kTile * CH / kThreads; ++it) {
                const int r = (tid + it * kThreads) / CH, ch = tid % CH;
                const int p = key0 + r;
                bool ok = p < end;
                size_t at = 0;
                if (ok) {
                    const int page = __ldg(table + p / a.c.ps);
                    ok = (unsigned)page < (unsigned)a.c.num_pages;
                    if (ok) at = (((size_t)page * a.c.Hkv + x.hk) * a.c.ps + p % a.c.ps) * D + ch * 8;
                    else s_bad[st] = j + 1;
                }
                cp_async16(dk + swz<D>(r, ch), a.k + at, ok);
                cp_async16(dv + swz<D>(r, ch), a.v + at, ok);
            }
            ld.next(a);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) load(j);

    const int rw = warp % RW, kw = warp / RW;
    uint32_t qa[KS][4];
    float o[D / 8][4], m[2], l[2];
    int pos[2];
    int start = cur.i;  // first tile of the entry in this run
    bool bad = false, fresh = true;
    Entry x;
    for (int j = 0; j < n; ++j) {
        cp_async_wait<kStages - 2>();
        __syncthreads();
        load(j + kStages - 1);
        const int st = j % kStages;
        bad |= s_bad[st] == j + 1;
        if (fresh) {
            fresh = false;
            x = get_entry(a, cur.e);
            start = cur.i;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = rw * 16 + (lane >> 2) + 8 * h;
                const bool ok = r < x.nt * a.G;
                pos[h] = ok ? x.pos0 + r / a.G : -1;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(
                    a.q + ((size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G) * D) + (lane & 3);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qa[ks][h] = ok ? __ldg(src + ks * 8) : 0u;
                    qa[ks][h + 2] = ok ? __ldg(src + ks * 8 + 4) : 0u;
                }
                m[h] = -INFINITY;
                l[h] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
        }
        unsigned long long mask;
        const int key0 = tile_of(cur, mask) + kw * KPW;
        const uint32_t sk = s0 + st * 2 * S::kTileBytes, sv = sk + S::kTileBytes;
        float s[KPW / 8][4];
#pragma unroll
        for (int i = 0; i < KPW / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int np = 0; np < KPW / 16; ++np) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4(b0, b1, b2, b3,
                        sk + swz<D>(kw * KPW + np * 16 + (lane & 7) + ((lane >> 4) << 3),
                                    ks * 2 + ((lane >> 3) & 1)));
                mma16816(s[2 * np], qa[ks], b0, b1);
                mma16816(s[2 * np + 1], qa[ks], b2, b3);
            }
        float mx[2] = {-INFINITY, -INFINITY}, mu[2];
        const int row = rw * 16 + (lane >> 2);
        // last key that each of the two rows sees
        const int see[2] = {(mask >> row) & 1 ? pos[0] : -1, (mask >> (row + 8)) & 1 ? pos[1] : -1};
#pragma unroll
        for (int i = 0; i < KPW / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int key = key0 + i * 8 + 2 * (lane & 3) + (k & 1);
                const float y = key > see[k >> 1] ? -INFINITY : s[i][k] * a.scale_log2;
                s[i][k] = y;
                mx[k >> 1] = fmaxf(mx[k >> 1], y);
            }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            const float mn = fmaxf(m[h], mx[h]);
            mu[h] = mn == -INFINITY ? 0.f : mn;
            const float f = fast_exp2(m[h] - mu[h]);
            m[h] = mn;
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                o[i][2 * h] *= f;
                o[i][2 * h + 1] *= f;
            }
        }
#pragma unroll
        for (int i = 0; i < KPW / 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                s[i][k] = fast_exp2(s[i][k] - mu[k >> 1]);
                l[k >> 1] += s[i][k];
            }
#pragma unroll
        for (int kk = 0; kk < KPW / 16; ++kk) {
            const uint32_t pa[4] = {pack_bf16(s[2 * kk][0], s[2 * kk][1]),
                                    pack_bf16(s[2 * kk][2], s[2 * kk][3]),
                                    pack_bf16(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                    pack_bf16(s[2 * kk + 1][2], s[2 * kk + 1][3])};
#pragma unroll
            for (int dp = 0; dp < D / 16; ++dp) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(b0, b1, b2, b3,
                          sv + swz<D>(kw * KPW + kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3),
                                      dp * 2 + (lane >> 4)));
                mma16816(o[2 * dp], pa, b0, b1);
                mma16816(o[2 * dp + 1], pa, b2, b3);
            }
        }
        const bool end = cur.i == cur.T - 1;
        if (end || j == n - 1) {
            // ---- the entry's rows leave this run ----
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int at = kw * ROWS + row + 8 * h;
                if ((lane & 3) == 0) {
                    s_m[at] = m[h];
                    s_l[at] = l[h];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2 *>(comb + at * D + i * 8 + 2 * (lane & 3)) =
                        make_float2(o[i][2 * h], o[i][2 * h + 1]);
            }
            bad = __syncthreads_or(bad);
            const bool whole = end && start == 0;
            const int slot = cta * 2 + (start == 0 ? 1 : 0);
            if (tid == 0) {
                if (start == 0) a.c_first[cur.e] = cta;
                if (end) a.c_last[cur.e] = cta;
                if (bad) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
            }
            for (int id = tid; id < x.nt * a.G * CH; id += kThreads) {
                const int r = id / CH, d = id % CH * 8;
                float M = -INFINITY, Lsum = 0.f, acc[8];
#pragma unroll
                for (int w = 0; w < KW; ++w) M = fmaxf(M, s_m[w * ROWS + r]);
                const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
                for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    const float f = fast_exp2(s_m[w * ROWS + r] - ref);
                    Lsum = fmaf(s_l[w * ROWS + r], f, Lsum);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        acc[k] = fmaf(comb[(w * ROWS + r) * D + d + k], f, acc[k]);
                }
                if (whole) {
                    const size_t at = (size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G;
                    const float inv = bad ? 0.f : 1.f / Lsum;
                    uint4 w;
                    uint32_t *pw = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        pw[k] = bad ? 0u : pack_bf16(acc[2 * k] * inv, acc[2 * k + 1] * inv);
                    *reinterpret_cast<uint4 *>(a.out + at * D + d) = w;
                    if (d == 0)
                        a.lse[at] = bad ? -INFINITY : (M + log2f(Lsum)) * 0.69314718055994530942f;
                } else {
                    float *dst = a.part_o + ((size_t)slot * ROWS + r) * D + d;
                    *reinterpret_cast<float4 *>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                    *reinterpret_cast<float4 *>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
                    if (d == 0) a.part_ml[(size_t)slot * ROWS + r] = make_float2(M, bad ? -1.f : Lsum);
                }
            }
            bad = false;
            fresh = true;
        }
        cur.next(a);
    }
    cp_async_wait<0>();
}

// Joins the partial sums of the entries that several CTAs worked on, and clears
// the rows of refused sequences.  A warp per row.
template <int D>
__global__ void __launch_bounds__(kThreads) merge_kernel(Attn a) {
    const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Entry x = get_entry(a, e);
    if (x.state == kSeqEmpty) return;
    const int nrows = x.nt * a.G;
    const bool none = x.state == kSeqBad || get_tiles(a, e) == 0;
    if (x.state == kSeqBad && threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
    int first = 0, last = 0;
    if (!none) {
        first = a.c_first[e];
        last = a.c_last[e];
        if (first == last) return;  // written by that CTA
    }
    for (int r = warp; r < nrows; r += kThreads / 32) {
        const size_t at = (size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G;
        float M = -INFINITY, L = 0.f;
        bool bad = none;
        if (!none)
            for (int c = first + lane; c <= last; c += 32) {
                const float2 ml = a.part_ml[(size_t)(2 * c + (c == first)) * a.rows + r];
                bad |= ml.y < 0.f;
                M = fmaxf(M, ml.x);
            }
        bad = __any_sync(0xffffffffu, bad);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float ref = M == -INFINITY ? 0.f : M;
        float acc[D / 32];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) acc[k] = 0.f;
        if (!bad)
            for (int c = first; c <= last; ++c) {
                const size_t p = (size_t)(2 * c + (c == first)) * a.rows + r;
                const float2 ml = a.part_ml[p];
                const float f = fast_exp2(ml.x - ref);
                L = fmaf(ml.y, f, L);
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    acc[k] = fmaf(a.part_o[p * D + lane * (D / 32) + k], f, acc[k]);
            }
        const float inv = 1.f / L;
#pragma unroll
        for (int k = 0; k < D / 32; k += 2)
            *reinterpret_cast<uint32_t *>(a.out + at * D + lane * (D / 32) + k) =
                bad ? 0u : pack_bf16(acc[k] * inv, acc[k + 1] * inv);
        if (lane == 0) a.lse[at] = bad ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    }
}

template <int D, int RW>
cudaError_t launch(const Attn &a, cudaStream_t st) {
    const int bytes = (int)RowsSmem<D>::kBytes;
    cudaError_t rc = cudaFuncSetAttribute(rows_kernel<D, RW>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (rc != cudaSuccess) return rc;
    rows_kernel<D, RW><<<a.ctas, kThreads, bytes, st>>>(a);
    rc = cudaGetLastError();
    if (rc != cudaSuccess) return rc;
    merge_kernel<D><<<a.n_ent, kThreads, 0, st>>>(a);
    note_launches(2);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Attn &a, cudaStream_t st) {
    return a.rows == 16 ? launch<D, 1>(a, st) : a.rows == 32 ? launch<D, 2>(a, st) : launch<D, 4>(a, st);
}

}  // namespace

cudaError_t launch_rows(const Attn &a, cudaStream_t st) {
    return a.D == 64 ? launch_d<64>(a, st) : launch_d<128>(a, st);
}

// ----------------------------------------------------------------------------
// host side of the call
// ----------------------------------------------------------------------------
namespace {

size_t scratch(Attn *a, void *base) {
    size_t off = 0;
    auto take = [&](size_t bytes) -> void * {
        void *p = base ? static_cast<char *>(base) + off : nullptr;
        off = (off + bytes + 255) & ~size_t(255);
        return p;
    };
    const size_t n = a->n_ent;
    // entries, CTAs and rows that share partial sums
    const size_t ents = a->chunk ? (size_t)a->w_cap * a->c.Hkv : n;
    const size_t parts = 2 * (size_t)a->ctas * (a->chunk ? kJobRows : a->rows);
    if (a->dense || !a->chunk) {
        a->c_first = static_cast<int *>(take(4 * ents));
        a->c_last = static_cast<int *>(take(4 * ents));
        a->part_ml = static_cast<float2 *>(take(sizeof(float2) * parts));
        a->part_o = static_cast<float *>(take(sizeof(float) * parts * a->D));
    }
    if (!a->dense) {
        a->tiles = static_cast<int *>(take(4 * n));
        a->ublk = static_cast<int *>(take(4 * n * a->ucap));
        a->umask = static_cast<unsigned long long *>(take(8 * n * a->ucap));
    }
    if (a->chunk) {
        a->own_off = static_cast<int *>(take(4 * ((size_t)a->c.num_seqs + 1)));
        a->unit_off = static_cast<long long *>(take(8 * ((size_t)a->w_cap + 1)));
    }
    if (a->chunk && !a->dense) {
        const size_t lists = (size_t)a->c.num_seqs * a->n_max * a->c.Hkv;
        const size_t slots = (size_t)a->c.total * a->Hq * (a->km1 + 1);
        a->counts = static_cast<int *>(take(4 * lists));
        a->list_off = static_cast<int *>(take(4 * (lists + 1)));
        a->jobs = static_cast<int2 *>(take(8 * (size_t)a->job_cap));
        a->n_jobs = static_cast<int *>(take(4));
        a->list = static_cast<int *>(take(4 * (size_t)a->list_cap));
        a->ubase = static_cast<int *>(take(4 * n * a->ucap));
        a->part_h = static_cast<__half *>(take(sizeof(__half) * slots * a->D));
        a->part_s = static_cast<float4 *>(take(sizeof(float4) * slots));
    }
    return off;
}

// Sizes of a call whose cache has been checked (a->c is filled).
int make_attn(Attn *a, int Hq, int D, int topk) {
    if (Hq < 1 || topk < 1 || Hq % a->c.Hkv) return MOBA_ERR_INVALID_ARG;
    a->Hq = Hq;
    a->G = Hq / a->c.Hkv;
    if (a->G > kMaxRows || Hq > 65535) return MOBA_ERR_UNSUPPORTED;
    a->D = D;
    a->topk = topk;
    const int bs = a->c.bs;
    const long long n_max = ((long long)a->c.max_pages * a->c.ps + bs - 1) / bs;
    a->dense = topk >= n_max;
    a->km1 = a->dense ? 0 : topk - 1;
    if (!a->dense && (a->km1 > kMaxPastSlots || n_max > kMaxBlocks)) return MOBA_ERR_UNSUPPORTED;
    const long long rows = (long long)a->c.max_new * a->G;
    a->rows = rows <= 16 && a->G <= 16 ? 16 : rows <= 32 && a->G <= 32 ? 32 : 64;
    a->tt = a->rows / a->G;
    a->tps = (a->c.max_new + a->tt - 1) / a->tt;
    const long long n_ent = (long long)a->c.num_seqs * a->tps * a->c.Hkv;
    if (n_ent >= (1ll << 31)) return MOBA_ERR_UNSUPPORTED;
    a->n_ent = (int)n_ent;
    a->tpb = bs / kTile;
    a->ctas = sm_count();
    a->n_max = (int)(n_max < (1 << 30) ? n_max : 1 << 30);
    // more rows than an entry holds go to the tcgen05 kernel, where row numbers
    // (token, head of the group) and lists are 32-bit
    const long long lists = a->dense ? 0 : (long long)a->c.num_seqs * n_max * a->c.Hkv;
    a->list_cap = (long long)a->c.total * Hq * a->km1;
    a->chunk = rows > kMaxRows && (long long)a->c.total * a->G < (1ll << 26) &&
               lists < (1ll << 30) && a->list_cap < (1ll << 31);
    if (a->chunk) {
        const long long w0 = (long long)a->c.num_seqs * ((rows + kJobRows - 1) / kJobRows);
        const long long w1 = (long long)a->c.total * a->G / kJobRows + a->c.num_seqs;
        a->w_cap = (int)(w0 < w1 ? w0 : w1);
        a->job_cap = a->list_cap / kJobRows + (lists < a->list_cap ? lists : a->list_cap) + 1;
        if ((long long)a->w_cap * a->c.Hkv >= (1ll << 30)) return MOBA_ERR_UNSUPPORTED;
    }
    const long long ucap = (long long)a->rows * (a->km1 + (a->chunk ? 0 : 1));
    a->ucap = a->dense ? 0 : (int)(ucap < n_max ? (ucap > 0 ? ucap : 1) : n_max);
    a->scale_log2 = (float)(1.4426950408889634 / __builtin_sqrt((double)D));
    return MOBA_OK;
}

}  // namespace
}  // namespace paged
}  // namespace moba

using namespace moba;
using namespace moba::paged;

MOBA_EXPORT size_t moba_paged_attn_workspace_size(int num_seqs, int total, int max_new, int Hq,
                                                  int Hkv, int D, int page_size, int max_pages,
                                                  int block_size, int topk) {
    Attn a = {};
    // any non-null, aligned addresses: only the sizes matter here
    const void *some = reinterpret_cast<const void *>(256);
    if (make_cache(&a.c, some, some, nullptr, static_cast<const int32_t *>(some),
                   static_cast<const int32_t *>(some), static_cast<const int32_t *>(some), num_seqs,
                   total, max_new, Hkv, D, 1, page_size, max_pages, block_size) != MOBA_OK ||
        make_attn(&a, Hq, D, topk) != MOBA_OK)
        return 0;
    return scratch(&a, nullptr);
}

MOBA_EXPORT int moba_paged_attn(const void *q, const void *k_pages, const void *v_pages,
                                const float *kbar_pages, const int32_t *page_table,
                                const int32_t *cu_new, const int32_t *cache_lens, void *out,
                                float *lse, int32_t *idx, int num_seqs, int total, int max_new,
                                int Hq, int Hkv, int D, int num_pages, int page_size,
                                int max_pages, int block_size, int topk, void *workspace,
                                size_t workspace_bytes, void *stream) {
    if (!q || !out || !lse) return MOBA_ERR_INVALID_ARG;
    Attn a = {};
    int rc = make_cache(&a.c, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens, num_seqs,
                        total, max_new, Hkv, D, num_pages, page_size, max_pages, block_size);
    if (rc == MOBA_OK) rc = make_attn(&a, Hq, D, topk);
    if (rc != MOBA_OK) return rc;
    if (misaligned16(q) || misaligned16(out) ||
        ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(idx)) & 3))
        return MOBA_ERR_INVALID_ARG;
    if (a.km1 > 0 && !kbar_pages) return MOBA_ERR_INVALID_ARG;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k_pages);
    a.v = static_cast<const __nv_bfloat16 *>(v_pages);
    a.kbar = kbar_pages;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.lse = lse;
    a.idx = idx;
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
    cudaError_t e = cudaSuccess;
    if (a.chunk && !a.dense)
        e = cudaMemsetAsync(a.counts, 0, 4 * (size_t)num_seqs * a.n_max * Hkv, st);
    if (e == cudaSuccess) e = launch_gate(a, st);
    if (e == cudaSuccess && a.chunk) e = launch_plan(a, st);
    if (e == cudaSuccess) e = a.chunk ? launch_chunk(a, st) : launch_rows(a, st);
    if (own) {
        const cudaError_t f = cudaFreeAsync(own, st);
        if (e == cudaSuccess) e = f;
    }
    return cuda_result(e);
}
