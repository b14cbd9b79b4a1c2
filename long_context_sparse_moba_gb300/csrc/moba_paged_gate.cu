// moba_paged_gate.cu -- block selection of new tokens over a paged cache.
//
// Pages: "Moonshot MoBA paper explained" (gsyq.cn/news/227272) sections 3.1
// and 4.1 (scores by the mean key, future blocks masked, the top_k of the sorted
// scores) and "MOBA mixture of block attention for server-side long context"
// (hncyxsy.com/news/197418) section 3 (the own block forced).
//
// 64 pooled keys at a time are split into two bf16 terms (hi + lo) and scored on
// the tensor cores, q being bf16 already.  A score errs by at most 2^-18 |q||k|
// for the split (two roundings of 2^-9) and 2 D roundings of at most 2^-23 |q||k| for
// the sums.  The accumulators go straight into the selection: the four lanes of a
// row hold 16 scores each as integers in the scores' order, their low 7 bits replaced
// by the score's place (2^-16 of the score), and each round of a maximum over the
// lanes yields the next best; the topk + 1 best of the tiles before compete again.
// (A list kept by insertion costs several times the instructions.)
// A score is off by E = 1.1 (2^-18 + D 2^-22) |q| max|k| at most (plus terms for values
// so small that they underflow) and by 2^-16 of itself.  Where the last kept and the
// first dropped score are more than twice that apart, the selection is settled (a
// lower score's upper end is lower too); the other rows (one in a hundred on random
// keys, all of them when keys tie) are decided by a warp with 64-bit scores, so that
// the selection is the one of 64-bit arithmetic: scores of the topk best by fp32 where
// the next one lies as far below the boundary, else of all blocks within three times
// that of it.
//
// gate_kernel: one CTA per entry (up to 64 query rows that share a kv head); then
// the blocks that any row selected are listed, each with the rows that did: the
// attention kernel reads a block once for all rows of the entry.
// chunk_gate_kernel: chunks of many rows, 128 rows to a CTA; a row takes its
// place in the list of each block that it selected.
// Bound: latency and mma.sync, not bytes.  A step of 8 sequences with 63 past
// blocks takes 10 to 17 us, a chunk of 4096 tokens x 32 heads of 128 over 64 blocks
// 54 us: of a CTA's 38 K cycles, three CTAs side by side on an SM, 6 K bring the
// pooled keys in, 12 K score (8 cycles an MMA on each of the SM's four parts), 5 K
// rank, 8 K go to near ties and 6 K to the lists.  (2.5 rows a ns; the prefill gate's
// tcgen05 scores reach 6.)  Three CTAs an SM leave chunk_gate_kernel 80 registers: with
// heads of 128 it spills 96 bytes up to top-k 3 and 156 up to 7, and its 1032 CTAs are
// two waves and a quarter.  From top-k 8 on the ranks take up to 236 registers, one CTA.
#include "moba_mma.cuh"
#include "moba_paged_attn.cuh"
#include "moba_select.cuh"

namespace moba {
namespace paged {
namespace {

using namespace mma;

constexpr int kThreads = 128;

// dynamic shared memory of the gate, in order
struct GateSmem {
    uint32_t hi, lo, sel, bits, rank, mask, bytes;
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

// The same among n given blocks, in any order; four at a time, their loads and
// sums side by side (one after the other they took a fifth of the kernel).
template <int D>
__device__ __noinline__ int pick64_of(const Attn &a, int hk, const int *table, const __nv_bfloat16 *qr,
                                      const int *ids, int n) {
    constexpr int U = 4, DL = D / 32;
    const int lane = threadIdx.x & 31, ppb = a.c.bs / a.c.ps;
    double q[DL];
#pragma unroll
    for (int d = 0; d < DL; ++d) q[d] = (double)__bfloat162float(qr[32 * d + lane]);
    double best = -INFINITY;
    int who = sel::kEmpty;
    for (int i0 = 0; i0 < n; i0 += U) {
        int c[U];
        float k[U][DL];
        double s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            c[u] = i0 + u < n ? ids[i0 + u] : sel::kEmpty;
            const int page = i0 + u < n ? __ldg(table + (c[u] + 1) * ppb - 1) : -1;
            if ((unsigned)page >= (unsigned)a.c.num_pages) c[u] = sel::kEmpty;
#pragma unroll
            for (int d = 0; d < DL; ++d)
                k[u][d] = c[u] == sel::kEmpty
                              ? 0.f
                              : __ldg(a.kbar + ((size_t)page * a.c.Hkv + hk) * D + 32 * d + lane);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u] = 0.0;
#pragma unroll
            for (int d = 0; d < DL; ++d) s[u] = fma(q[d], (double)k[u][d], s[u]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int u = 0; u < U; ++u) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (c[u] == sel::kEmpty) continue;  // (every lane alike)
            if (s[u] != s[u]) s[u] = -INFINITY;
            const int at = __popc(__ballot_sync(
                0xffffffffu, who != sel::kEmpty && (best > s[u] || (best == s[u] && who < c[u]))));
            const double pb = __shfl_up_sync(0xffffffffu, best, 1);
            const int pw = __shfl_up_sync(0xffffffffu, who, 1);
            if (lane > at) {
                best = pb;
                who = pw;
            } else if (lane == at) {
                best = s[u];
                who = c[u];
            }
        }
    }
    return who;
}

// The best scores of a row so far, spread over the row's four lanes: rank r with
// lane r % 4, place r / 4.  `key`: the score's bits in integer order, the low 7
// bits cleared.
constexpr int kNone = (int)0x80000000;
template <int NS>
struct Best {
    int key[NS], blk[NS];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            key[i] = kNone;
            blk[i] = sel::kEmpty;
        }
    }
    // the 16 scores of this lane (blocks cb + 8 j + 2 (lane % 4) + k, those from `own`
    // on left out) against the ranks so far; `want` ranks are kept
    __device__ __forceinline__ void rank(const float (&acc)[8][4], int h, int cb, int own, int want) {
        const int lane = threadIdx.x & 31;
        int v[16], old[NS];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int at = (j >> 1) * 8 + 2 * (lane & 3) + (j & 1);
            const int x = __float_as_int(acc[j >> 1][2 * h + (j & 1)]);
            // NaN as -inf; below zero the order of the bits is turned around
            const int y = (x & 0x7fffffff) > 0x7f800000 ? (int)0x807fffff : x ^ ((x >> 31) & 0x7fffffff);
            v[j] = cb + at < own ? ((y & ~127) | at) : kNone;
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            old[i] = blk[i];
            key[i] = blk[i] == sel::kEmpty ? kNone : key[i] | (64 + 4 * i + (lane & 3));
        }
        int nkey[NS], nblk[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            nkey[i] = kNone;
            nblk[i] = sel::kEmpty;
#pragma unroll 1
            for (int l = 0; l < 4; ++l) {
                if (4 * i + l >= want) break;
                int m = key[0];
#pragma unroll
                for (int k = 1; k < NS; ++k) m = max(m, key[k]);
#pragma unroll
                for (int j = 0; j < 16; ++j) m = max(m, v[j]);
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
                // its block: of this tile, or of the rank that it had
                const int id = m & 127, was = (id - 64) >> 2;
                int b = old[0];
#pragma unroll
                for (int k = 1; k < NS; ++k) b = was == k ? old[k] : b;
                b = __shfl_sync(0xffffffffu, b, (lane & 28) | (id & 3));
                if (id < 64) b = cb + id;
                if ((lane & 3) == l) {
                    nkey[i] = m & ~127;
                    nblk[i] = m == kNone ? sel::kEmpty : b;
                }
                if (m != kNone) {
#pragma unroll
                    for (int k = 0; k < NS; ++k) key[k] = key[k] == m ? kNone : key[k];
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = v[j] == m ? kNone : v[j];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            key[i] = nkey[i];
            blk[i] = nblk[i];
        }
    }
    // the score and the block of a rank, to all four lanes
    __device__ __forceinline__ float score(int r, int &b) const {
        const int lane = threadIdx.x & 31;
        int k = key[0];
        b = blk[0];
#pragma unroll
        for (int i = 1; i < NS; ++i) {
            k = (r >> 2) == i ? key[i] : k;
            b = (r >> 2) == i ? blk[i] : b;
        }
        k = __shfl_sync(0xffffffffu, k, (lane & 28) | (r & 3));
        b = __shfl_sync(0xffffffffu, b, (lane & 28) | (r & 3));
        return b == sel::kEmpty ? -INFINITY : __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
    }
};

// Rows left to 64-bit scores.
template <int ROWS>
struct Unsure {
    int n, row[ROWS], few[ROWS];
    float from[ROWS];
};

// A row's ranks into sel[0 .. km1], and whether its selection is settled.  All
// four lanes of a row (r < 0: of no row).
template <int D, int NS, int ROWS>
__device__ __forceinline__ void decide(const Best<NS> &best, int r, int own, int km1, float q2,
                                       float knmax, int *sel, Unsure<ROWS> &un) {
    const int lane = threadIdx.x & 31;
    int b;
    const float kept = best.score(km1 - 1, b), dropped = best.score(km1, b);
    const float next = best.score(km1 + 1, b);
    if (r < 0 || own <= km1) return;
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (4 * i + (lane & 3) <= km1) sel[r * (km1 + 1) + 4 * i + (lane & 3)] = best.blk[i];
    // (the squares of values below 1e-22 vanish in fp32, products below 1e-38 in the
    // scores: far below any real score, the additions keep the bound a bound)
    constexpr float kBound = 1.1f * (0x1p-18f + D * 0x1p-22f), kPlace = 0x1p-16f;
    const float base = fmaf(sqrtf(q2 + 1e-36f), knmax * kBound, 1e-35f);
    const float err = fmaf(fmaxf(fabsf(kept), fabsf(dropped)), kPlace, base);
    if ((lane & 3) == 0 && !(kept - dropped > 2.f * err)) {
        const int u = atomicAdd(&un.n, 1);
        un.row[u] = r;
        un.from[u] = kept - 3.f * err;
        un.few[u] = b == sel::kEmpty ||  // (there is no next one)
                    next < kept - 2.f * fmaf(fmaxf(fabsf(kept), fabsf(next)), kPlace, base);
    }
}

// The pages that hold the pooled keys of blocks [cb, cb + 64): -1 from c_end on,
// and for a page outside the pool.
__device__ __forceinline__ void load_pages(const Attn &a, const int *table, int cb, int c_end,
                                           int *s_page, int *s_bad) {
    const int tid = threadIdx.x, ppb = a.c.bs / a.c.ps;
    if (tid < kTile) {
        const int page = cb + tid < c_end ? __ldg(table + (cb + tid + 1) * ppb - 1) : -1;
        const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
        s_page[tid] = ok ? page : -1;
        if (cb + tid < c_end && !ok) *s_bad = 1;
    }
}

// Those pooled keys, split into bf16 hi + lo tiles (zeros where there is no page),
// and their largest norm into s_knmax.  T threads, FLY loads of a thread in flight.
// Between two barriers.
template <int D, int T, int FLY>
__device__ __forceinline__ void load_pooled(const Attn &a, int hk, const int *s_page, int *s_knmax,
                                            uint8_t *hi, uint8_t *lo) {
    constexpr int LR = D / 4;  // lanes per pooled key, four values each
    constexpr int NR = kTile / (T / LR);
    const int tid = threadIdx.x;
    constexpr int HALF = NR > FLY ? FLY : NR;
    float kn = 0.f;
#pragma unroll
    for (int i0 = 0; i0 < NR; i0 += HALF) {
        float4 f[HALF];
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
            const int page = s_page[(i0 + i) * (T / LR) + tid / LR];
            f[i] = page < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : __ldg(reinterpret_cast<const float4 *>(
                                        a.kbar + ((size_t)page * a.c.Hkv + hk) * D) + tid % LR);
        }
#pragma unroll
        for (int i = 0; i < HALF; ++i) {
            const int r = (i0 + i) * (T / LR) + tid / LR;
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
            *reinterpret_cast<uint2 *>(hi + at) = *reinterpret_cast<uint2 *>(h);
            *reinterpret_cast<uint2 *>(lo + at) = *reinterpret_cast<uint2 *>(l);
#pragma unroll
            for (int o = LR / 2; o > 0; o >>= 1) n2 += __shfl_xor_sync(0xffffffffu, n2, o);
            kn = n2 > kn || n2 != n2 ? n2 : kn;
        }
    }
    // a NaN norm has the largest bits of all
    if (tid % LR == 0) atomicMax(s_knmax, __float_as_int(fabsf(sqrtf(kn + 1e-36f))));
}

// Scores of this warp's 16 rows with the 64 pooled keys.
template <int D>
__device__ __forceinline__ void score_tile(const uint32_t (&qa)[D / 16][4], uint32_t s_hi,
                                           uint32_t s_lo, float (&acc)[8][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
#pragma unroll
    for (int term = 0; term < 2; ++term) {
        const uint32_t base = term ? s_lo : s_hi;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
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
}

// Two rows of q as MMA operands (nullptr: zeros) and their squared norms.
template <int D>
__device__ __forceinline__ void load_q(const __nv_bfloat16 *q0, const __nv_bfloat16 *q1,
                                       uint32_t (&qa)[D / 16][4], float (&q2)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(h ? q1 : q0) + (threadIdx.x & 3);
        const bool live = (h ? q1 : q0) != nullptr;
        q2[h] = 0.f;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t u = live ? __ldg(src + ks * 8 + 4 * k) : 0u;
                qa[ks][h + 2 * k] = u;
                const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
                q2[h] = fmaf(f.x, f.x, fmaf(f.y, f.y, q2[h]));
            }
        q2[h] += __shfl_xor_sync(0xffffffffu, q2[h], 1);
        q2[h] += __shfl_xor_sync(0xffffffffu, q2[h], 2);
    }
}

// A row's selection by 64-bit scores into sel[0 .. km1); a warp.
template <int D>
__device__ __forceinline__ void settle(const Attn &a, int hk, const int *table, const __nv_bfloat16 *qr,
                                       int own, int few, float from, int *sel) {
    const int lane = threadIdx.x & 31, km1 = a.km1;
    int who = few ? pick64_of<D>(a, hk, table, qr, sel, min(km1 + 1, own))
                  : pick64<D>(a, hk, table, qr, own, from);
    // should the bound not have left enough: from the lowest score on
    if (__any_sync(0xffffffffu, lane < km1 && who == sel::kEmpty))
        who = pick64<D>(a, hk, table, qr, own, -INFINITY);
    __syncwarp();
    if (lane < km1) sel[lane] = who;
}

// (four CTAs an SM where 128 registers hold the ranks: the compiler's own choice of 168
// left three; 32 and 64 sequences of 32 kv heads over 64 blocks of 128, k 6, 108 and
// 196 us, against 116 and 205)
template <int D, int NS>
__global__ void __launch_bounds__(kThreads, NS > 2 ? 0 : 4) gate_kernel(Attn a, int words) {
    constexpr int KS = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_bad, s_knmax, s_count, s_page[kTile];
    __shared__ Unsure<kMaxRows> s_un;
    let_next();
    const GateSmem L = gate_smem(D, words, a.ucap, a.km1);
    int *sel = reinterpret_cast<int *>(smem + L.sel);  // [row][km1 + 1]
    unsigned *bits = reinterpret_cast<unsigned *>(smem + L.bits);
    int *rank = reinterpret_cast<int *>(smem + L.rank);
    unsigned long long *mask = reinterpret_cast<unsigned long long *>(smem + L.mask);
    const int e = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Entry x = get_entry(a, e);
    const int bs = a.c.bs, km1 = a.km1, G = a.G;
    const int nrows = x.nt * G;
    if (x.state != kSeqOk) {  // (refused rows are cleared by the attention kernel)
        if (tid == 0) a.tiles[e] = 0;
        return;
    }
    const int pos_last = x.pos0 + x.nt - 1, c_own = pos_last / bs;
    const int *table = a.c.table + (size_t)x.b * a.c.max_pages;
    if (tid == 0) {
        s_bad = 0;
        s_knmax = 0;
        s_un.n = 0;
    }
    for (int i = tid; i < words; i += kThreads) bits[i] = 0;
    __syncthreads();
    const bool scored = km1 > 0 && c_own > km1;
    const int ss = km1 + 1;  // of a row's blocks in `sel`
    auto q_of = [&](int r) -> const __nv_bfloat16 * {
        return a.q + ((size_t)(x.row0 + r / G) * a.Hq + x.hk * G + r % G) * D;
    };
    auto own_of = [&](int r) -> int { return (x.pos0 + r / G) / bs; };
    if (scored) {
        load_pages(a, table, 0, c_own, s_page, &s_bad);  // (in flight with q)
        // this warp's 16 rows of q as MMA operands, and each row's norm
        uint32_t qa[KS][4];
        float q2[2];
        const int rq = warp * 16 + (lane >> 2);
        load_q<D>(rq < nrows ? q_of(rq) : nullptr, rq + 8 < nrows ? q_of(rq + 8) : nullptr, qa, q2);
        const int ci[2] = {rq < nrows ? own_of(rq) : 0, rq + 8 < nrows ? own_of(rq + 8) : 0};
        Best<NS> best[2];
        best[0].clear();
        best[1].clear();
        const uint32_t s_hi = smem_u32(smem + L.hi), s_lo = smem_u32(smem + L.lo);
        for (int cb = 0; cb < c_own; cb += kTile) {
            if (cb > 0) {
                __syncthreads();  // (the tile before has been read)
                load_pages(a, table, cb, c_own, s_page, &s_bad);
            }
            __syncthreads();
            load_pooled<D, kThreads, 16>(a, x.hk, s_page, &s_knmax, smem + L.hi, smem + L.lo);
            __syncthreads();
            if (warp * 16 < nrows) {
                float acc[8][4];
                score_tile<D>(qa, s_hi, s_lo, acc);
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (warp * 16 + 8 * h < nrows) best[h].rank(acc, h, cb, ci[h], km1 + 2);
            }
        }
        if (warp * 16 < nrows)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                decide<D>(best[h], rq + 8 * h < nrows ? rq + 8 * h : -1, ci[h], km1, q2[h],
                       __int_as_float(s_knmax), sel, s_un);
        __syncthreads();
        // rows that the error bound leaves open: a warp each
        for (int u = warp; u < s_un.n; u += kThreads / 32) {
            const int r = s_un.row[u];
            settle<D>(a, x.hk, table, q_of(r), own_of(r), s_un.few[u], s_un.from[u], sel + r * ss);
        }
        __syncthreads();
    }
    const bool bad = scored && s_bad;
    // each row's selection, ascending (a row with few past blocks takes them all)
    const bool row_ok = tid < nrows;
    const int row = tid, ci = row_ok ? own_of(row) : 0;
    if (row_ok) {
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
            atomicOr(bits + (ci >> 5), 1u << (ci & 31));
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
    if (row_ok) {
        const int n = min(km1, ci);
        for (int i = 0; i <= n; ++i) {
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
    if (tid == 0) a.tiles[e] = (count - 1) * a.tpb + (pos_last - c_own * bs) / kTile + 1;
}

// ----------------------------------------------------------------------------
// chunks of many rows
// ----------------------------------------------------------------------------
constexpr int kChunkRows = 128, kChunkThreads = 256;
constexpr int kPlaces = 1024;  // blocks whose rows are counted in shared memory

__host__ __device__ constexpr int chunk_gate_smem(int D, int km1) {
    return 2 * kTile * D * 2 + 4 * kChunkRows * (2 * km1 + 1);
}

// Zeros where the gate counts: the gate runs beside it up to its first count (a
// memset before the gate cost the chunk 2 us).
__global__ void __launch_bounds__(kChunkThreads) zero_kernel(int *p, long long n) {
    let_next();
    for (long long i = (long long)blockIdx.x * kChunkThreads + threadIdx.x; i < n;
         i += (long long)gridDim.x * kChunkThreads)
        p[i] = 0;
}

template <int D, int NS>
__global__ void __launch_bounds__(kChunkThreads, NS > 2 ? 1 : 3) chunk_gate_kernel(Attn a) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_bad, s_knmax, s_page[kTile], s_place[kPlaces];
    __shared__ Unsure<kChunkRows> s_un;
    uint8_t *const hi = smem, *const lo = smem + kTile * D * 2;
    int *sel = reinterpret_cast<int *>(smem + 2 * kTile * D * 2);  // [row][km1 + 1]
    let_next();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int tile;
    const int hk = blockIdx.x % a.c.Hkv, b = a.c.tile_of(blockIdx.x / a.c.Hkv, a.G, kChunkRows, 1, tile);
    const int bs = a.c.bs, km1 = a.km1, G = a.G, ss = km1 + 1;
    Seq s;
    const int state = a.c.seq(b, s);
    if (state != kSeqOk || tile < 0 || (long long)tile * kChunkRows >= (long long)s.n * G) {
        after_previous();  // (refused rows are cleared by the plan)
        return;
    }
    const int r0 = tile * kChunkRows, nrows = min(kChunkRows, s.n * G - r0);
    const int row0 = s.row0 * G + r0;  // row = row0 + r: token row / G, head row % G
    const int pdelta = s.len - s.n - s.row0;  // position of a row = its token + pdelta
    const int c_own = ((row0 + nrows - 1) / G + pdelta) / bs;
    const int *table = a.c.table + (size_t)b * a.c.max_pages;
    if (tid == 0) {
        s_bad = 0;
        s_knmax = 0;
        s_un.n = 0;
    }
    auto q_of = [&](int r) -> const __nv_bfloat16 * {
        const int row = row0 + r;
        return a.q + ((size_t)(row / G) * a.Hq + hk * G + row % G) * D;
    };
    auto own_of = [&](int r) -> int { return ((row0 + r) / G + pdelta) / bs; };
    const bool scored = km1 > 0 && c_own > km1;
    if (scored) {
        float q2[2] = {0.f, 0.f};
        const int rq = warp * 16 + (lane >> 2);  // the quad's first row
        const __nv_bfloat16 *q0 = rq < nrows ? q_of(rq) : nullptr;
        const __nv_bfloat16 *q1 = rq + 8 < nrows ? q_of(rq + 8) : nullptr;
        const int ci[2] = {rq < nrows ? own_of(rq) : 0, rq + 8 < nrows ? own_of(rq + 8) : 0};
        Best<NS> best[2];
        best[0].clear();
        best[1].clear();
        const uint32_t s_hi = smem_u32(hi), s_lo = smem_u32(lo);
        for (int cb = 0; cb < c_own; cb += kTile) {
            __syncthreads();  // (the tile before has been read)
            load_pages(a, table, cb, c_own, s_page, &s_bad);
            __syncthreads();
            load_pooled<D, kChunkThreads, 4>(a, hk, s_page, &s_knmax, hi, lo);
            __syncthreads();
            if (warp * 16 < nrows) {
                float acc[8][4];
                {   // (q read again for each tile: its registers are free for the ranks)
                    uint32_t qa[D / 16][4];
                    load_q<D>(q0, q1, qa, q2);
                    score_tile<D>(qa, s_hi, s_lo, acc);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) best[h].rank(acc, h, cb, ci[h], km1 + 2);
            }
        }
        if (warp * 16 < nrows)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                decide<D>(best[h], rq + 8 * h < nrows ? rq + 8 * h : -1, ci[h], km1, q2[h],
                       __int_as_float(s_knmax), sel, s_un);
        __syncthreads();
        for (int u = warp; u < s_un.n; u += kChunkThreads / 32) {
            const int r = s_un.row[u];
            settle<D>(a, hk, table, q_of(r), own_of(r), s_un.few[u], s_un.from[u], sel + r * ss);
        }
    }
    __syncthreads();
    const bool bad = scored && s_bad;
    if (bad && tid == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
    // each row's selection, ascending
    const int own = tid < nrows ? own_of(tid) : 0, n = tid < nrows ? min(km1, own) : 0;
    const int row = row0 + tid;
    int *mine = sel + tid * ss;
    if (own > km1) {
        for (int i = 1; i < n; ++i) {
            const int v = mine[i];
            int j = i - 1;
            for (; j >= 0 && mine[j] > v; --j) mine[j + 1] = mine[j];
            mine[j + 1] = v;
        }
    } else {
        for (int i = 0; i < n; ++i) mine[i] = i;
    }
    if (a.idx && tid < nrows) {
        int32_t *dst = a.idx + ((size_t)(row / G) * a.Hq + hk * G + row % G) * a.topk;
        for (int i = 0; i < a.topk; ++i) dst[i] = bad || i > n ? -1 : i < n ? mine[i] : own;
    }
    after_previous();
    // its places in the blocks' lists: counted in shared memory first, then one
    // global addition per block and CTA (an addition per row and block waits a
    // third of the kernel for the few hundred counters that all rows share)
    int *counts = a.counts + (size_t)b * a.n_max * a.c.Hkv + hk;
    int2 *out = a.sel + ((size_t)hk * a.c.total * G + row) * km1;
    const bool counted = c_own <= kPlaces;
    int *at = sel + kChunkRows * ss + tid * km1;  // the row's places among this CTA's
    if (counted) {
        for (int c = tid; c < c_own; c += kChunkThreads) s_place[c] = 0;
        __syncthreads();
        if (!bad)
            for (int i = 0; i < n; ++i) at[i] = atomicAdd(s_place + mine[i], 1);
        __syncthreads();
        for (int c = tid; c < c_own; c += kChunkThreads)
            if (s_place[c]) s_place[c] = atomicAdd(counts + (size_t)c * a.c.Hkv, s_place[c]);
        __syncthreads();
    }
    if (tid >= nrows) return;
    if (hk == 0 && row % G == 0) a.tok[row / G] = row / G + pdelta + 1;
    const int list0 = b * a.n_max * a.c.Hkv + hk;
    for (int i = 0; i < km1; ++i) {
        const int c = bad ? kSelBad : i < n ? mine[i] : -1;
        const int place = c < 0 ? 0 : counted ? s_place[c] + at[i] : atomicAdd(counts + (size_t)c * a.c.Hkv, 1);
        out[i] = make_int2(c < 0 ? c : list0 + c * a.c.Hkv, place);
    }
}

// The selection where topk covers every block: all of them.
constexpr int kFillTokens = 16;  // of a CTA

__global__ void __launch_bounds__(kThreads) fill_kernel(Attn a) {
    let_next();
    int tile;
    const int b = a.c.tile_of(blockIdx.x, 1, kFillTokens, 1, tile);
    Seq s;
    // (refused rows are cleared by the kernels that follow)
    if (a.c.seq(b, s) != kSeqOk || tile < 0 || (long long)tile * kFillTokens >= s.n) return;
    const int t0 = tile * kFillTokens, nt = min(kFillTokens, s.n - t0);
    const long long per = (long long)a.Hq * a.topk;  // of a token
    for (long long i = threadIdx.x; i < nt * per; i += kThreads) {
        const int t = t0 + (int)(i / per), j = (int)(i % a.topk);
        const int own = (s.len - s.n + t) / a.c.bs;
        a.idx[(s.row0 + t0) * per + i] = j <= own ? j : -1;
    }
}

template <int D, int NS>
cudaError_t launch(const Attn &a, cudaStream_t st) {
    const int words = (int)(((long long)a.c.max_pages * a.c.ps / a.c.bs) / 32 + 1);
    const int bytes = (int)gate_smem(D, words, a.ucap, a.km1).bytes;
    constexpr int kMost = kMaxRows * (kMaxPastSlots + 1);
    const cudaError_t rc = allow_smem<gate_kernel<D, NS>>(
        (int)gate_smem(D, kMaxBlocks / 32 + 1, kMost, kMaxPastSlots).bytes);
    if (rc != cudaSuccess) return rc;
    gate_kernel<D, NS><<<a.n_ent, kThreads, bytes, st>>>(a, words);
    note_launches(1);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Attn &a, cudaStream_t st) {
    // ranks: the kept ones, the first dropped one and the next, four to a place
    if (a.km1 <= 2) return launch<D, 1>(a, st);
    if (a.km1 <= 6) return launch<D, 2>(a, st);
    if (a.km1 <= 14) return launch<D, 4>(a, st);
    return launch<D, 9>(a, st);
}

template <int D, int NS>
cudaError_t launch_c(const Attn &a, cudaStream_t st) {
    const cudaError_t rc = allow_smem<chunk_gate_kernel<D, NS>>(chunk_gate_smem(D, kMaxPastSlots));
    if (rc != cudaSuccess) return rc;
    note_launches(1);
    return launch_after(chunk_gate_kernel<D, NS>, (unsigned)(a.c.tile_slots(a.G, kChunkRows, 1) * a.c.Hkv),
                        kChunkThreads, chunk_gate_smem(D, a.km1), st, a);
}

template <int D>
cudaError_t launch_cd(const Attn &a, cudaStream_t st) {
    if (a.km1 <= 2) return launch_c<D, 1>(a, st);
    if (a.km1 <= 6) return launch_c<D, 2>(a, st);
    if (a.km1 <= 14) return launch_c<D, 4>(a, st);
    return launch_c<D, 9>(a, st);
}

}  // namespace

cudaError_t launch_gate(const Attn &a, cudaStream_t st) {
    if (a.dense) {
        if (!a.idx) return cudaSuccess;
        fill_kernel<<<(unsigned)a.c.tile_slots(1, kFillTokens, 1), kThreads, 0, st>>>(a);
        note_launches(1);
        return cudaGetLastError();
    }
    return a.D == 64 ? launch_d<64>(a, st) : launch_d<128>(a, st);
}

cudaError_t launch_chunk_gate(const Attn &a, cudaStream_t st) {
    const long long n = (long long)a.c.num_seqs * a.n_max * a.c.Hkv + a.c.total;  // counts and tok
    const long long ctas = (n + 4 * kChunkThreads - 1) / (4 * kChunkThreads);
    zero_kernel<<<(unsigned)(ctas < 4 * a.ctas ? ctas : 4 * a.ctas), kChunkThreads, 0, st>>>(a.counts, n);
    note_launches(1);
    const cudaError_t rc = cudaGetLastError();
    if (rc != cudaSuccess) return rc;
    return a.D == 64 ? launch_cd<64>(a, st) : launch_cd<128>(a, st);
}

}  // namespace paged
}  // namespace moba
