// moba_paged_gate.cu -- block selection of new tokens over a paged cache.
//
// Pages: "Moonshot MoBA paper explained" (gsyq.cn/news/227272) sections 3.1
// and 4.1 (scores by the mean key, future blocks masked, the top_k of the sorted
// scores) and "MOBA mixture of block attention for server-side long context"
// (hncyxsy.com/news/197418) section 3 (the own block forced).
//
// One CTA per entry (up to 64 query rows that share a kv head).  64 pooled keys
// at a time are split into two bf16 terms (hi + lo) and scored on the tensor
// cores, q being bf16 already; a thread per row keeps the topk best.
// A score errs by at most 2^-16 |q||k| for the split and 256 roundings of at
// most 2^-23 |q||k| for the sums, less than E = 2^-14 |q| max|k| together (plus
// a term for pooled keys so small that lo underflows).  Where the last kept and
// the first dropped score are more than 2 E apart the selection is settled;
// the other rows (about one in a hundred on random keys, all of them when keys
// tie) are decided by a warp with 64-bit scores, so that the selection is the
// one of 64-bit arithmetic: scores of the topk best by fp32 where the next one
// lies 2 E below the boundary, else of all blocks within 3 E of it.
// Then the blocks that any row selected are listed, each with the rows that
// did: the attention kernel reads a block once for all rows of the entry.  For
// chunks of many rows the own blocks stay out of it, and each block's count of
// rows over all entries is taken, for lists of the rows that selected it.
#include "moba_mma.cuh"
#include "moba_paged_attn.cuh"
#include "moba_select.cuh"

namespace moba {
namespace paged {
namespace {

using namespace mma;

constexpr int kThreads = 128;
constexpr int kScStride = kTile + 1;

// dynamic shared memory of the gate, in order
struct GateSmem {
    uint32_t hi, lo, sc, sel, bits, rank, mask, bytes;
};
__host__ __device__ inline GateSmem gate_smem(int D, int words, int ucap, int km1) {
    GateSmem s;
    uint32_t o = 0;
    s.hi = o;
    o += kTile * D * 2;
    s.lo = o;
    o += kTile * D * 2;
    s.mask = o;
    o += 8 * ucap;
    s.sc = o;
    o += 4 * kMaxRows * kScStride;
    s.sel = o;
    o += 4 * kMaxRows * (km1 + 1);
    s.bits = o;
    o += 4 * words;
    s.rank = o;
    o += 4 * words;
    s.bytes = o;
    return s;
}

// One row's best blocks by 64-bit scores, among its cr past blocks whose fp32
// score is not below `from`: lane i returns the i-th best (kEmpty: there are no
// so many).  Blocks come in ascending order and move ahead of no equal score.
// A warp; every lane holds the same arguments.
template <int D>
__device__ __noinline__ int pick64(const Attn &a, int hk, const int *table, const __nv_bfloat16 *qr,
                                   int cr, float from) {
    const int lane = threadIdx.x & 31, ppb = a.c.bs / a.c.ps;
    double best = -INFINITY;
    int who = sel::kEmpty;
    for (int cb = 0; cb < cr; cb += 32) {
        const int c = cb + lane;
        bool near = false;
        int page = -1;
        if (c < cr) {
            page = __ldg(table + (c + 1) * ppb - 1);
            if ((unsigned)page < (unsigned)a.c.num_pages)
                near = !(sel::exact_score<D>(qr, a.kbar + ((size_t)page * a.c.Hkv + hk) * D) < from);
        }
        unsigned todo = __ballot_sync(0xffffffffu, near);
        while (todo) {
            const int j = __ffs(todo) - 1;
            todo &= todo - 1;
            const int pg = __shfl_sync(0xffffffffu, page, j);
            const float *kb = a.kbar + ((size_t)pg * a.c.Hkv + hk) * D;
            double s = 0.0;
#pragma unroll
            for (int d = 0; d < D; d += 32)
                s = fma((double)__bfloat162float(qr[d + lane]), (double)__ldg(kb + d + lane), s);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (s != s) s = -INFINITY;
            const int at = __popc(__ballot_sync(0xffffffffu, who != sel::kEmpty && best >= s));
            const double pb = __shfl_up_sync(0xffffffffu, best, 1);
            const int pw = __shfl_up_sync(0xffffffffu, who, 1);
            if (lane > at) {
                best = pb;
                who = pw;
            } else if (lane == at) {
                best = s;
                who = cb + j;
            }
        }
    }
    return who;
}

// The same among n given blocks, in any order.
template <int D>
__device__ __noinline__ int pick64_of(const Attn &a, int hk, const int *table, const __nv_bfloat16 *qr,
                                      const int *ids, int n) {
    const int lane = threadIdx.x & 31, ppb = a.c.bs / a.c.ps;
    double best = -INFINITY;
    int who = sel::kEmpty;
    for (int i = 0; i < n; ++i) {
        const int c = ids[i], page = __ldg(table + (c + 1) * ppb - 1);
        if ((unsigned)page >= (unsigned)a.c.num_pages) continue;
        const float *kb = a.kbar + ((size_t)page * a.c.Hkv + hk) * D;
        double s = 0.0;
#pragma unroll
        for (int d = 0; d < D; d += 32)
            s = fma((double)__bfloat162float(qr[d + lane]), (double)__ldg(kb + d + lane), s);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (s != s) s = -INFINITY;
        const int at = __popc(__ballot_sync(
            0xffffffffu, who != sel::kEmpty && (best > s || (best == s && who < c))));
        const double pb = __shfl_up_sync(0xffffffffu, best, 1);
        const int pw = __shfl_up_sync(0xffffffffu, who, 1);
        if (lane > at) {
            best = pb;
            who = pw;
        } else if (lane == at) {
            best = s;
            who = c;
        }
    }
    return who;
}

// insert (x, c) into a descending list; an equal score keeps the lower block first
template <int KCAP>
__device__ __forceinline__ void merge_insert(float (&ts)[KCAP], int (&ti)[KCAP], float x, int c) {
    bool ins = false;
#pragma unroll
    for (int s = 0; s < KCAP; ++s) {
        if (ins || x > ts[s] || ti[s] == sel::kEmpty || (x == ts[s] && c < ti[s])) {
            const float fs = ts[s];
            const int fi = ti[s];
            ts[s] = x;
            ti[s] = c;
            x = fs;
            c = fi;
            ins = true;
        }
    }
}

template <int D, int KCAP>
__global__ void __launch_bounds__(kThreads) gate_kernel(Attn a, int words) {
    constexpr int KS = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_bad, s_knmax, s_unsure, s_count, s_rows[kMaxRows], s_few[kMaxRows], s_page[kTile];
    __shared__ float s_floor[kMaxRows];
    let_next();
    const GateSmem L = gate_smem(D, words, a.ucap, a.km1);
    float *sc = reinterpret_cast<float *>(smem + L.sc);
    int *sel = reinterpret_cast<int *>(smem + L.sel);  // [row][km1 + 1]
    unsigned *bits = reinterpret_cast<unsigned *>(smem + L.bits);
    int *rank = reinterpret_cast<int *>(smem + L.rank);
    unsigned long long *mask = reinterpret_cast<unsigned long long *>(smem + L.mask);
    const int e = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Entry x = get_entry(a, e);
    const int bs = a.c.bs, km1 = a.km1, G = a.G;
    const int nrows = x.nt * G;
    if (x.state != kSeqOk) {
        if (tid == 0) a.tiles[e] = 0;
        if (x.state == kSeqBad && a.idx)
            for (int i = tid; i < nrows * a.topk; i += kThreads) {
                const int r = i / a.topk;
                a.idx[((size_t)(x.row0 + r / G) * a.Hq + x.hk * G + r % G) * a.topk + i % a.topk] = -1;
            }
        return;
    }
    const int pos_last = x.pos0 + x.nt - 1, c_own = pos_last / bs;
    const int *table = a.c.table + (size_t)x.b * a.c.max_pages;
    const int ppb = bs / a.c.ps;
    if (tid == 0) {
        s_bad = 0;
        s_knmax = 0;
        s_unsure = 0;
    }
    for (int i = tid; i < words; i += kThreads) bits[i] = 0;
    __syncthreads();
    // two threads to a row, for half the scores of a tile each
    const int row = tid >> 1, half = tid & 1;
    const bool row_ok = row < nrows;
    const int ci = row_ok ? (x.pos0 + row / G) / bs : 0;  // the row's own block
    const __nv_bfloat16 *qrow = a.q + ((size_t)(x.row0 + row / G) * a.Hq + x.hk * G + row % G) * D;
    const bool scored = km1 > 0 && c_own > km1;
    const int ss = km1 + 1;  // of a row's blocks in `sel`
    if (scored) {
        // this warp's 16 rows of q as MMA operands, and each row's norm
        uint32_t qa[KS][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = warp * 16 + (lane >> 2) + 8 * h;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                a.q + ((size_t)(x.row0 + r / G) * a.Hq + x.hk * G + r % G) * D) + (lane & 3);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                qa[ks][h] = r < nrows ? __ldg(src + ks * 8) : 0u;
                qa[ks][h + 2] = r < nrows ? __ldg(src + ks * 8 + 4) : 0u;
            }
        }
        float q2 = 0.f;
        if (row_ok)
#pragma unroll
            for (int d = 0; d < D / 2; d += 8) {
                const uint4 u = __ldg(reinterpret_cast<const uint4 *>(qrow + half * (D / 2) + d));
                const __nv_bfloat162 *p2 = reinterpret_cast<const __nv_bfloat162 *>(&u);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __bfloat1622float2(p2[i]);
                    q2 = fmaf(f.x, f.x, fmaf(f.y, f.y, q2));
                }
            }
        q2 += __shfl_xor_sync(0xffffffffu, q2, 1);
        float ts[KCAP];
        int ti[KCAP];
#pragma unroll
        for (int i = 0; i < KCAP; ++i) {
            ts[i] = -INFINITY;
            ti[i] = sel::kEmpty;
        }
        float worst = -INFINITY;
        const uint32_t s_hi = smem_u32(smem + L.hi), s_lo = smem_u32(smem + L.lo);
        for (int cb = 0; cb < c_own; cb += kTile) {
            // 64 pooled keys, four values a lane, split into hi + lo
            constexpr int LR = D / 4;  // lanes per pooled key
            constexpr int NR = kTile / (kThreads / LR);
            if (tid < kTile) {
                const int page = cb + tid < c_own ? __ldg(table + (cb + tid + 1) * ppb - 1) : -1;
                const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
                s_page[tid] = ok ? page : -1;
                if (cb + tid < c_own && !ok) s_bad = 1;
            }
            __syncthreads();
            float4 f[NR];
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int page = s_page[i * (kThreads / LR) + tid / LR];
                f[i] = page < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                                : __ldg(reinterpret_cast<const float4 *>(
                                            a.kbar + ((size_t)page * a.c.Hkv + x.hk) * D) + tid % LR);
            }
            float kn = 0.f;
#pragma unroll
            for (int i = 0; i < NR; ++i) {
                const int r = i * (kThreads / LR) + tid / LR;
                const float v[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
                __nv_bfloat16 h[4], l[4];
                float n2 = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    h[k] = __float2bfloat16(v[k]);
                    l[k] = __float2bfloat16(v[k] - __bfloat162float(h[k]));
                    n2 = fmaf(v[k], v[k], n2);
                }
                const uint32_t at = swz<D>(r, (tid % LR) >> 1) + (tid & 1) * 8;
                *reinterpret_cast<uint2 *>(smem + L.hi + at) = *reinterpret_cast<uint2 *>(h);
                *reinterpret_cast<uint2 *>(smem + L.lo + at) = *reinterpret_cast<uint2 *>(l);
#pragma unroll
                for (int o = LR / 2; o > 0; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
                kn = n2 > kn || n2 != n2 ? n2 : kn;
            }
            // a NaN norm has the largest bits of all
            if (tid % LR == 0) atomicMax(&s_knmax, __float_as_int(fabsf(sqrtf(kn))));
            __syncthreads();
            float acc[8][4];
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
            if (warp * 16 < nrows) {
#pragma unroll
                for (int term = 0; term < 2; ++term) {
                    const uint32_t base = term ? s_lo : s_hi;
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                        for (int np = 0; np < 4; ++np) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(b0, b1, b2, b3,
                                    base + swz<D>(np * 16 + (lane & 7) + ((lane >> 4) << 3),
                                                  ks * 2 + ((lane >> 3) & 1)));
                            mma16816(acc[2 * np], qa[ks], b0, b1);
                            mma16816(acc[2 * np + 1], qa[ks], b2, b3);
                        }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sc[(warp * 16 + (lane >> 2) + (i >> 1) * 8) * kScStride + j * 8 +
                           2 * (lane & 3) + (i & 1)] = acc[j][i];
            }
            __syncthreads();
            if (row_ok) {
                const int n = min(kTile / 2 * (half + 1), ci - cb);
                for (int k = kTile / 2 * half; k < n; ++k) {
                    float y = sc[row * kScStride + k];
                    if (y != y) y = -INFINITY;
                    if (y > worst || ti[KCAP - 1] == sel::kEmpty) {
                        sel::top_insert<KCAP>(ts, ti, KCAP, y, cb + k);
                        worst = ts[KCAP - 1];
                    }
                }
            }
        }
        // the other thread's list into the first one's
#pragma unroll
        for (int i = 0; i < KCAP; ++i) {
            const float y = __shfl_xor_sync(0xffffffffu, ts[i], 1);
            const int c = __shfl_xor_sync(0xffffffffu, ti[i], 1);
            if (half == 0 && c != sel::kEmpty) merge_insert<KCAP>(ts, ti, y, c);
        }
        if (row_ok && half == 0 && ci > km1) {
            float kept = 0.f, dropped = 0.f, next = 0.f;
            bool none = false;  // there is no next one, or it is not held
#pragma unroll
            for (int i = 0; i < KCAP; ++i) {
                if (i == km1 - 1) kept = ts[i];
                if (i == km1) dropped = ts[i];
                if (i == km1 + 1) {
                    next = ts[i];
                    none = ti[i] == sel::kEmpty;
                }
                if (i <= km1) sel[row * ss + i] = ti[i];
            }
            const float err = sqrtf(q2) * fmaf(__int_as_float(s_knmax), 6.103515625e-5f, 1e-34f);
            if (!(kept - dropped > 2.f * err)) {
                const int u = atomicAdd(&s_unsure, 1);
                s_rows[u] = row;
                s_floor[u] = kept - 3.f * err;
                s_few[u] = km1 + 1 < KCAP && (none || next < kept - 2.f * err);
            }
        }
        __syncthreads();
        // rows that the error bound leaves open: 64-bit scores of the blocks
        // near the boundary, blocks ascending; lane i holds the i-th best
        for (int u = warp; u < s_unsure; u += kThreads / 32) {
            const int r = s_rows[u];
            const int cr = (x.pos0 + r / G) / bs;
            const __nv_bfloat16 *qr = a.q + ((size_t)(x.row0 + r / G) * a.Hq + x.hk * G + r % G) * D;
            int who = s_few[u] ? pick64_of<D>(a, x.hk, table, qr, sel + r * ss, min(ss, cr))
                               : pick64<D>(a, x.hk, table, qr, cr, s_floor[u]);
            // should the bound not have left enough: from the lowest score on
            if (__any_sync(0xffffffffu, lane < km1 && who == sel::kEmpty))
                who = pick64<D>(a, x.hk, table, qr, cr, -INFINITY);
            __syncwarp();
            if (lane < km1) sel[r * ss + lane] = who;
        }
        __syncthreads();
    }
    const bool bad = scored && s_bad;
    // each row's selection, ascending (a row with few past blocks takes them all)
    if (row_ok && half == 0) {
        const int n = min(km1, ci);
        int *mine = sel + row * ss;
        if (ci > km1) {
            for (int i = 1; i < n; ++i) {
                const int v = mine[i];
                int j = i - 1;
                for (; j >= 0 && mine[j] > v; --j) mine[j + 1] = mine[j];
                mine[j + 1] = v;
            }
        } else {
            for (int i = 0; i < n; ++i) mine[i] = i;
        }
        if (!bad) {
            for (int i = 0; i < n; ++i) atomicOr(bits + (mine[i] >> 5), 1u << (mine[i] & 31));
            if (!a.chunk) atomicOr(bits + (ci >> 5), 1u << (ci & 31));
        }
        if (a.idx) {
            int32_t *dst = a.idx + ((size_t)(x.row0 + row / G) * a.Hq + x.hk * G + row % G) * a.topk;
            for (int i = 0; i < a.topk; ++i) dst[i] = bad || i > n ? -1 : i < n ? mine[i] : ci;
        }
    }
    __syncthreads();
    if (bad) {
        if (tid == 0) {
            a.tiles[e] = 0;
            atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        }
        return;
    }
    // the union: rank of each block among the selected ones, and its rows
    const int used = (c_own >> 5) + 1;
    if (warp == 0) {
        int run = 0;
        for (int w0 = 0; w0 < used; w0 += 32) {
            const int w = w0 + lane;
            const int n = w < used ? __popc(bits[w]) : 0;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (w < used) rank[w] = run + inc - n;
            run += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) s_count = run;
    }
    __syncthreads();
    const int count = s_count;
    for (int i = tid; i < count; i += kThreads) mask[i] = 0ull;
    __syncthreads();
    if (row_ok && half == 0) {
        const int n = min(km1, ci);
        for (int i = 0; i < n + (a.chunk ? 0 : 1); ++i) {
            const int c = i < n ? sel[row * ss + i] : ci;
            const int at = rank[c >> 5] + __popc(bits[c >> 5] & ((1u << (c & 31)) - 1u));
            atomicOr(mask + at, 1ull << row);
        }
    }
    __syncthreads();
    int *ublk = a.ublk + (size_t)e * a.ucap;
    unsigned long long *umask = a.umask + (size_t)e * a.ucap;
    for (int w = tid; w < used; w += kThreads) {
        unsigned b = bits[w];
        int at = rank[w];
        while (b) {
            ublk[at++] = w * 32 + __ffs(b) - 1;
            b &= b - 1;
        }
    }
    for (int i = tid; i < count; i += kThreads) umask[i] = mask[i];
    if (!a.chunk) {
        if (tid == 0) a.tiles[e] = (count - 1) * a.tpb + (pos_last - c_own * bs) / kTile + 1;
        return;
    }
    // this entry's place in the list of each block that its rows selected
    if (tid == 0) a.tiles[e] = count + 1;
    __syncthreads();
    for (int i = tid; i < count; i += kThreads)
        a.ubase[(size_t)e * a.ucap + i] =
            atomicAdd(a.counts + ((size_t)x.b * a.n_max + ublk[i]) * a.c.Hkv + x.hk, __popcll(mask[i]));
}

// The selection where topk covers every block: all of them.
__global__ void __launch_bounds__(kThreads) fill_kernel(Attn a) {
    let_next();
    const Entry x = get_entry(a, blockIdx.x);
    if (x.state == kSeqEmpty) return;
    const long long n = (long long)x.nt * a.G * a.topk;
    for (long long i = threadIdx.x; i < n; i += kThreads) {
        const int r = (int)(i / a.topk), j = (int)(i % a.topk);
        const int ci = (x.pos0 + r / a.G) / a.c.bs;
        a.idx[((size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G) * a.topk + j] =
            x.state == kSeqOk && j <= ci ? j : -1;
    }
}

template <int D, int KCAP>
cudaError_t launch(const Attn &a, cudaStream_t st) {
    const int words = (int)(((long long)a.c.max_pages * a.c.ps / a.c.bs) / 32 + 1);
    const int bytes = (int)gate_smem(D, words, a.ucap, a.km1).bytes;
    constexpr int kMost = kMaxRows * (kMaxPastSlots + 1);
    const cudaError_t rc = allow_smem<gate_kernel<D, KCAP>>(
        (int)gate_smem(D, kMaxBlocks / 32 + 1, kMost, kMaxPastSlots).bytes);
    if (rc != cudaSuccess) return rc;
    gate_kernel<D, KCAP><<<a.n_ent, kThreads, bytes, st>>>(a, words);
    note_launches(1);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Attn &a, cudaStream_t st) {
    // the kept ones, the first dropped one, and the next where there is room
    if (a.km1 <= 2) return launch<D, 4>(a, st);
    if (a.km1 <= 6) return launch<D, 8>(a, st);
    if (a.km1 <= 14) return launch<D, 16>(a, st);
    return launch<D, 32>(a, st);
}

}  // namespace

cudaError_t launch_gate(const Attn &a, cudaStream_t st) {
    if (a.dense) {
        if (!a.idx) return cudaSuccess;
        fill_kernel<<<a.n_ent, kThreads, 0, st>>>(a);
        note_launches(1);
        return cudaGetLastError();
    }
    return a.D == 64 ? launch_d<64>(a, st) : launch_d<128>(a, st);
}

}  // namespace paged
}  // namespace moba
