// moba_paged_rows.cu -- attention of a few query rows (up to 64 that share a kv
// head: the heads of a decode step, or of a few new tokens) over a paged cache, and
// the host side of the call.
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
// One warp brings the pages in by TMA, 128 KB or more in flight per SM: each of
// its lanes looks up the pages of one of the next 32 tiles, then they issue in
// turn.  CW warps attend: 16 rows each, RW of them side by side for the rows,
// the KW = CW / RW sets of them taking the tiles of the run in turn (stages are a
// multiple of KW, so a stage always belongs to the same set: a set that skipped
// phases of a stage's barrier could take an old phase for its own); they join
// through shared memory at the end of an entry's part.  Scores and outputs on
// mma.sync; one pass with running maximum and sum in 32 bits; P is rounded to
// bf16 for the second product, as the prefill kernels do: relative to 64 bits outputs
// err by 0.0022, of which the result's own rounding is 0.0016.  (A second bf16 term of P
// brings that back to 0.0016 and costs 3 % over all blocks, about 5 % with selection.)
// Waits on mbarriers are bounded as in the other kernels; a warp that gives up
// still joins the barrier of the part, where all warps agree to leave.
// Measured (heads of 128): 16 sequences of up to 49152 tokens, 32 / 8 heads, all blocks
// 312 us, 6.5 TB/s, 0.96 of the copy rate; 8 sequences, 32 heads, three blocks of
// 512 each 41 us, 5.1 TB/s.
#include "moba_mma.cuh"
#include "moba_paged_attn.cuh"
#include "moba_ptx.cuh"

namespace moba {
namespace paged {
namespace {

using ptx::Ctl;

constexpr int kParts = 4;  // part descriptors in flight

struct Part {
    int valid, e;
    int n;            // tiles
    int start, last;  // the part holds the entry's first, its last tile
    int pad[3];
};
struct Info {         // of a tile, beside its stage
    unsigned long long mask;
    int key0, nv;     // first key, keys that some row sees
    int bad, pad;
};

template <int D, int CW>
struct RowsSmem {
    static constexpr int NB = D / 64;
    static constexpr int kStages = 4 * (128 / D);
    static constexpr uint32_t kBox = kTile * 128;
    static constexpr uint32_t kTileBytes = NB * kBox;                // K or V
    static constexpr uint32_t kComb = kStages * 2 * kTileBytes;      // [CW * 16][D] fp32
    static constexpr uint32_t kInfo = kComb + CW * 16 * D * 4;
    static constexpr uint32_t kPart = kInfo + kStages * sizeof(Info);
    static constexpr uint32_t kBars = kPart + kParts * sizeof(Part);  // full, empty, part full, part empty
    static constexpr uint32_t kBytes = kBars + (2 * kStages + 2 * kParts) * 8 + 1024;
    static_assert(kBytes + 2048 <= 227 * 1024, "shared memory per CTA");
};

struct RowsArgs {
    Attn a;
    int psh;  // log2(page size)
    long long wait_limit;
};

// The rows of an entry without tiles, whose selection met a page outside the
// pool.  True: the entry is a refused sequence's.
template <int D>
__device__ __noinline__ bool clear_entry(const Attn &a, int e) {
    const Entry x = get_entry(a, e);
    if (x.state != kSeqOk) return x.state == kSeqBad;
    for (int r = 0; r < x.nt * a.G; ++r) {
        const size_t at = (size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G;
        a.lse[at] = -INFINITY;
        for (int d = 0; d < D; d += 8)
            *reinterpret_cast<uint4 *>(a.out + at * D + d) = make_uint4(0, 0, 0, 0);
    }
    return false;
}
// The refused sequences among this CTA's entries, one kv head's rows at a time.
__device__ __noinline__ void clear_sequences(const Attn &a) {
    for (int e = blockIdx.x; e < a.n_ent; e += gridDim.x) {
        const Entry x = get_entry(a, e);
        if (x.state != kSeqBad) continue;
        if (threadIdx.x == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        Seq s;
        a.c.seq(x.b, s);
        clear_refused(a, s, x.hk * a.G, a.G, threadIdx.x, blockDim.x);
    }
}

template <int D, int RW, int CW>
__global__ void __launch_bounds__(32 * (CW + 1), 1)
    rows_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const __grid_constant__ RowsArgs ra) {
    using S = RowsSmem<D, CW>;
    using mma::fast_exp2;
    using mma::ldsm_x4;
    using mma::ldsm_x4_t;
    using mma::mma16816;
    using mma::pack_bf16;
    constexpr int KS = D / 16, KW = CW / RW, ST = S::kStages;
    constexpr int kThreads = 32 * (CW + 1);
    constexpr int CH = D / 8;
    const Attn &a = ra.a;
    extern __shared__ uint8_t smem_raw[];
    __shared__ long long s_warp[CW + 1], s_base;
    __shared__ int s_e0, s_leave[CW], s_badw[CW];
    __shared__ int s_abort;
    __shared__ float s_m[CW * 16], s_l[CW * 16];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const uint32_t raw = ptx::saddr(smem_raw);
    const uint32_t s0 = (raw + 1023u) & ~1023u;
    uint8_t *smem = smem_raw + (s0 - raw);
    float *comb = reinterpret_cast<float *>(smem + S::kComb);
    Info *info = reinterpret_cast<Info *>(smem + S::kInfo);
    Part *parts = reinterpret_cast<Part *>(smem + S::kPart);
    auto full = [&](int s) { return s0 + S::kBars + 8u * s; };
    auto empty = [&](int s) { return s0 + S::kBars + 8u * (ST + s); };
    auto pfull = [&](int s) { return s0 + S::kBars + 8u * (2 * ST + s); };
    auto pempty = [&](int s) { return s0 + S::kBars + 8u * (2 * ST + kParts + s); };
    Ctl ctl{&s_abort, a.status, ra.wait_limit};

    // ---- this CTA's run of the tiles of all entries ----
    const int per = (a.n_ent + kThreads - 1) / kThreads;
    const int lo = min(tid * per, a.n_ent), hi = min(lo + per, a.n_ent);
    long long sum = 0;
    bool refused = false;
    after_previous();
    let_next();
    for (int e = lo; e < hi; ++e) {
        const int T = get_tiles(a, e);
        sum += T;
        if (T == 0 && e % (int)gridDim.x == cta) refused |= clear_entry<D>(a, e);
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[warp] = inc;
    if (tid == 0) {
        for (int s = 0; s < ST; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), RW);
        }
        for (int s = 0; s < kParts; ++s) {
            ptx::mbar_init(pfull(s), 1);
            ptx::mbar_init(pempty(s), CW);
        }
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    if (__syncthreads_or(refused)) clear_sequences(a);
    long long before = inc - sum, total = 0;
#pragma unroll
    for (int w = 0; w <= CW; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    // at least one tile each, so that an entry's runs are those of adjacent CTAs
    const long long runs = total < (long long)gridDim.x ? total : (long long)gridDim.x;
    if (cta >= runs) {
        if (tid == 0) a.c_open[cta] = -1;
        return;
    }
    const long long u0 = total * cta / runs, u1 = total * (cta + 1) / runs;
    if (u0 >= before && u0 < before + sum) {
        int e = lo;
        long long p = before;
        for (int t; u0 >= p + (t = get_tiles(a, e)); ++e) p += t;
        s_e0 = e;
        s_base = p;
    }
    __syncthreads();

    if (warp == CW) {
        // ================= pages =================
        const int n = (int)(u1 - u0), ps = a.c.ps, box = min(ps, kTile);
        int e = s_e0, i = (int)(u0 - s_base);  // where the batch starts
        int np = 0;                            // parts so far
        bool go = true;
        for (int t0 = 0; go && t0 < n; t0 += 32) {
            // lane: tile t0 + lane of the run
            const int t = t0 + lane;
            int le = e, li = i + lane, T = 0;
            if (t < n)
                while (li >= (T = get_tiles(a, le))) {
                    li -= T;
                    ++le;
                }
            Entry x;
            Info f;
            f.mask = ~0ull;
            int pages[kTile / 16] = {0, 0, 0, 0};
            f.bad = 0;
            f.pad = 0;
            f.key0 = f.nv = 0;
            if (t < n) {
                x = get_entry(a, le);
                if (a.dense) {
                    f.key0 = li * kTile;
                } else {
                    const int u = li / a.tpb;
                    f.mask = a.umask[(size_t)le * a.ucap + u];
                    f.key0 = a.ublk[(size_t)le * a.ucap + u] * a.c.bs + (li - u * a.tpb) * kTile;
                }
                f.nv = min(kTile, x.pos0 + x.nt - f.key0);
                const int *table = a.c.table + (size_t)x.b * a.c.max_pages;
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    if (k * box < f.nv) {
                        const int page = __ldg(table + ((f.key0 + k * box) >> ra.psh));
                        const bool ok = (unsigned)page < (unsigned)a.c.num_pages;
                        f.bad |= !ok;
                        // (some memory of the pool for a page outside it: its rows are dropped)
                        pages[k] = ((ok ? page : 0) * a.c.Hkv + x.hk) * ps + ((f.key0 + k * box) & (ps - 1));
                    }
            }
            const bool starts = t < n && (li == 0 || t == 0);
            const unsigned ballot = __ballot_sync(0xffffffffu, starts);
            const int pi = np + __popc(ballot & ((1u << lane) - 1u));
            for (int k = 0; k < 32 && t0 + k < n; ++k) {
                if (lane == k && go) {
                    if (starts) {
                        const int s = pi % kParts;
                        if (pi >= kParts) go = ptx::wait_bar(pempty(s), (pi / kParts - 1) & 1, ctl);
                        if (go) {
                            Part p;
                            p.valid = 1;
                            p.e = le;
                            p.n = min(T - li, n - t);
                            p.start = li == 0;
                            p.last = li + p.n == T;
                            p.pad[0] = p.pad[1] = p.pad[2] = 0;
                            parts[s] = p;
                            ptx::mbar_arrive(pfull(s));
                        }
                    }
                    const int st = t % ST;
                    if (go && t >= ST) go = ptx::wait_bar(empty(st), (t / ST - 1) & 1, ctl);
                    if (go) {
                        info[st] = f;
                        const int boxes = (f.nv + box - 1) / box;
                        ptx::mbar_expect_tx(full(st), (uint32_t)(boxes * box) * 256u * S::NB);
                        const uint32_t dk = s0 + st * 2 * S::kTileBytes;
#pragma unroll
                        for (int j = 0; j < kTile / 16; ++j)
                            if (j < boxes) {
#pragma unroll
                                for (int v = 0; v < 2; ++v)
#pragma unroll
                                    for (int b = 0; b < S::NB; ++b)
                                        asm volatile(
                                            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::"
                                            "complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                                                dk + v * S::kTileBytes + b * S::kBox +
                                                (uint32_t)(j * box) * 128u),
                                            "l"(reinterpret_cast<uint64_t>(v ? &tmap_v : &tmap_k)),
                                            "r"(full(st)), "r"(b * 64), "r"(pages[j])
                                            : "memory");
                            }
                    }
                }
                go = __shfl_sync(0xffffffffu, (int)go, k) != 0;
            }
            np += __popc(ballot);
            // the tile behind the batch
            const int last = min(31, n - 1 - t0);
            e = __shfl_sync(0xffffffffu, le, last);
            i = __shfl_sync(0xffffffffu, li, last) + 1;
        }
        if (go && lane == 0) {
            const int s = np % kParts;
            if (np < kParts || ptx::wait_bar(pempty(s), (np / kParts - 1) & 1, ctl)) {
                parts[s].valid = 0;
                ptx::mbar_arrive(pfull(s));
            }
        }
        if (!go && lane == 0) {
            // copies in flight land before the CTA ends: each stage's last phase
            for (int s = 0; s < ST; ++s)
                for (int ph = 0; ph < 2; ++ph) ptx::drain_bar(full(s), ph, ra.wait_limit / 8);
        }
        return;
    }

    // ================= attention =================
    const int rw = warp % RW, kw = warp / RW;
    const int row = rw * 16 + (lane >> 2);
    int tbase = 0, open = -1;
    for (int np = 0;; ++np) {
        const int s = np % kParts;
        bool ok = __all_sync(0xffffffffu, ptx::wait_bar(pfull(s), (np / kParts) & 1, ctl));
        Part part;
        part.valid = 0;
        if (ok) {
            part = parts[s];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(pempty(s));
        }
        const bool leave = !ok || !part.valid;
        uint32_t qa[KS][4];
        float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        int pos[2] = {-1, -1};
        bool bad = false;
        Entry x;
        x.nt = 0;
        if (!leave) {
            x = get_entry(a, part.e);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = row + 8 * h;
                const bool live = r < x.nt * a.G;
                pos[h] = live ? x.pos0 + r / a.G : -1;  // -1: no row, whose scores do not matter
                const uint32_t *src = reinterpret_cast<const uint32_t *>(
                    a.q + ((size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G) * D) + (lane & 3);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qa[ks][h] = live ? __ldg(src + ks * 8) : 0u;
                    qa[ks][h + 2] = live ? __ldg(src + ks * 8 + 4) : 0u;
                }
            }
#pragma unroll
            for (int i = 0; i < D / 8; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
            static_assert(ST % KW == 0, "a stage belongs to one set of warps");
            for (int t = tbase + (kw - tbase % KW + KW) % KW; t < tbase + part.n; t += KW) {
                const int st = t % ST;
                if (!__all_sync(0xffffffffu, ptx::wait_fast(full(st), (t / ST) & 1, ctl))) {
                    ok = false;
                    break;
                }
                const Info f = info[st];
                const uint32_t sk = s0 + st * 2 * S::kTileBytes, sv = sk + S::kTileBytes;
                bad |= f.bad != 0;
                if (f.nv < kTile) {
                    // keys that no row sees may never have been written: zeros in V
                    for (int z = lane; z < (kTile - f.nv) * 8 * S::NB; z += 32) {
                        const int b = z / ((kTile - f.nv) * 8), w = z % ((kTile - f.nv) * 8);
                        ptx::st_shared_v4(sv + b * S::kBox + f.nv * 128 + w * 16, 0, 0, 0, 0);
                    }
                    ptx::fence_proxy_async();
                    __syncwarp();
                }
                float sc[8][4];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[j][k] = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = j * 16 + (lane & 7) + ((lane >> 4) << 3);
                        const int c = ks * 2 + ((lane >> 3) & 1);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4(b0, b1, b2, b3,
                                sk + (c >> 3) * S::kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                        mma16816(sc[2 * j], qa[ks], b0, b1);
                        mma16816(sc[2 * j + 1], qa[ks], b2, b3);
                    }
                // last key that each of the two rows sees
                int see[2];
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    see[h] = pos[h] < 0 ? 0x7fffffff : (f.mask >> (row + 8 * h)) & 1 ? pos[h] : -1;
                float mx[2] = {-INFINITY, -INFINITY}, mu[2];
                const bool open = f.key0 + kTile - 1 <= min(see[0], see[1]);
                if (__all_sync(0xffffffffu, open)) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k >> 1] = fmaxf(mx[k >> 1], sc[j][k]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int key = f.key0 + j * 8 + 2 * (lane & 3) + (k & 1);
                            if (key > see[k >> 1]) sc[j][k] = -INFINITY;
                            mx[k >> 1] = fmaxf(mx[k >> 1], sc[j][k]);
                        }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * a.scale_log2;
                }
                if (__any_sync(0xffffffffu, mx[0] > m[0] || mx[1] > m[1])) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mn = fmaxf(m[h], mx[h]);
                        const float r = fast_exp2(m[h] - (mn == -INFINITY ? 0.f : mn));
                        m[h] = mn;
                        l[h] *= r;
#pragma unroll
                        for (int j = 0; j < D / 8; ++j) {
                            o[j][2 * h] *= r;
                            o[j][2 * h + 1] *= r;
                        }
                    }
                }
                mu[0] = m[0] == -INFINITY ? 0.f : m[0];
                mu[1] = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sc[j][k] = fast_exp2(fmaf(sc[j][k], a.scale_log2, -mu[k >> 1]));
                        l[k >> 1] += sc[j][k];
                    }
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const uint32_t pa[4] = {pack_bf16(sc[2 * kk][0], sc[2 * kk][1]),
                                            pack_bf16(sc[2 * kk][2], sc[2 * kk][3]),
                                            pack_bf16(sc[2 * kk + 1][0], sc[2 * kk + 1][1]),
                                            pack_bf16(sc[2 * kk + 1][2], sc[2 * kk + 1][3])};
                    const int r = kk * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
                    for (int dp = 0; dp < D / 16; ++dp) {
                        const int c = dp * 2 + (lane >> 4);
                        uint32_t b0, b1, b2, b3;
                        ldsm_x4_t(b0, b1, b2, b3,
                                  sv + (c >> 3) * S::kBox + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                        mma16816(o[2 * dp], pa, b0, b1);
                        mma16816(o[2 * dp + 1], pa, b2, b3);
                    }
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(empty(st));
            }
            tbase += part.n;
            // ---- the entry's rows leave this run ----
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int at = warp * 16 + (lane >> 2) + 8 * h;
                if ((lane & 3) == 0) {
                    s_m[at] = m[h];
                    s_l[at] = l[h];
                }
#pragma unroll
                for (int i = 0; i < D / 8; ++i)
                    *reinterpret_cast<float2 *>(comb + at * D + i * 8 + 2 * (lane & 3)) =
                        make_float2(o[i][2 * h], o[i][2 * h + 1]);
            }
        }
        if (lane == 0) {
            s_leave[warp] = leave || !ok;
            s_badw[warp] = bad;
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * CW) : "memory");
        bool out = false;
        bad = false;
#pragma unroll
        for (int w = 0; w < CW; ++w) {
            out |= s_leave[w] != 0;
            bad |= s_badw[w] != 0;
        }
        if (out) break;  // every warp of the attention alike
        const bool whole = part.start && part.last;
        const int slot = cta * 2 + (part.start ? 1 : 0);
        if (tid == 0) {
            if (part.start && !part.last) open = part.e;
            if (part.last) a.c_last[part.e] = cta;
            if (bad) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        }
        for (int id = tid; id < x.nt * a.G * CH; id += 32 * CW) {
            const int r = id / CH, d = id % CH * 8;
            float M = -INFINITY, Lsum = 0.f, acc[8];
#pragma unroll
            for (int w = 0; w < KW; ++w) M = fmaxf(M, s_m[(w * RW + r / 16) * 16 + r % 16]);
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
                const int at = (w * RW + r / 16) * 16 + r % 16;
                const float f = fast_exp2(s_m[at] - ref);
                Lsum = fmaf(s_l[at], f, Lsum);
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(comb + at * D + d + k);
                    acc[k] = fmaf(v.x, f, acc[k]);
                    acc[k + 1] = fmaf(v.y, f, acc[k + 1]);
                    acc[k + 2] = fmaf(v.z, f, acc[k + 2]);
                    acc[k + 3] = fmaf(v.w, f, acc[k + 3]);
                }
            }
            if (whole) {
                const size_t at = (size_t)(x.row0 + r / a.G) * a.Hq + x.hk * a.G + r % a.G;
                const float inv = 1.f / Lsum;
                uint4 w;
                uint32_t *pw = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    pw[k] = bad ? 0u : pack_bf16(acc[2 * k] * inv, acc[2 * k + 1] * inv);
                *reinterpret_cast<uint4 *>(a.out + at * D + d) = w;
                if (d == 0)
                    a.lse[at] = bad ? -INFINITY : (M + log2f(Lsum)) * 0.69314718055994530942f;
            } else {
                float *dst = a.part_o + ((size_t)slot * a.rows + r) * D + d;
                *reinterpret_cast<float4 *>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
                *reinterpret_cast<float4 *>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
                if (d == 0) a.part_ml[(size_t)slot * a.rows + r] = make_float2(M, bad ? -1.f : Lsum);
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * CW) : "memory");  // before the next part's sums
    }
    if (tid == 0) a.c_open[cta] = open;
}

// Joins the partial sums of an entry (a row tile of a chunk) that starts in one
// CTA's run and ends in another's.  Few parts: a warp a row.  Many (a long cache
// of few heads): four warps a row, every fourth part each, joined in shared
// memory.  Four parts in flight.  A chunk's tile has 256 rows and seldom many
// parts, so a CTA takes 64 of them and looks the tile up once.
constexpr int kMergeThreads = 512, kFewParts = 8;
__host__ __device__ constexpr int merge_rows(bool chunk) { return chunk ? 64 : 4; }  // of a CTA

template <int D, bool CHUNK>
__global__ void __launch_bounds__(kMergeThreads) merge_runs_kernel(Attn a) {
    constexpr int V = D / 32, U = 4;
    __shared__ float s_acc[16][D], s_m[16], s_l[16];
    after_previous();
    const int first = blockIdx.x, e = a.c_open[first];
    if (e < 0) return;
    const int last = min(a.c_last[e], (int)gridDim.x - 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = CHUNK ? kJobRows : a.rows;
    const int W = last - first < kFewParts ? 1 : 4;  // warps to a row
    const int part = warp % W;
    Entry x;
    int row0 = 0, nrows, hk;
    if (CHUNK) {
        const int w = e / a.c.Hkv, b = seq_of_tile(a, w);
        Seq s;
        a.c.seq(b, s);
        const int r0 = (w - a.own_off[b]) * kJobRows;
        row0 = s.row0 * a.G + r0;
        nrows = min(kJobRows, s.n * a.G - r0);
        hk = e % a.c.Hkv;
    } else {
        x = get_entry(a, e);
        row0 = x.row0 * a.G;
        nrows = x.nt * a.G;
        hk = x.hk;
    }
    for (int r0 = 0; r0 < merge_rows(CHUNK); r0 += 16 / W) {
        const int r = blockIdx.y * merge_rows(CHUNK) + r0 + warp / W;
        const bool live = r < nrows && r0 + warp / W < merge_rows(CHUNK);
        float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        bool bad = false;
        if (live)
            for (int c0 = first + part; c0 <= last; c0 += W * U) {
                float2 ml[U];
                float v[U][V];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const int c = c0 + W * j;
                    ml[j] = make_float2(-INFINITY, 0.f);
                    if (c <= last) {
                        const size_t p = (size_t)(2 * c + (c == first)) * R + r;
                        ml[j] = a.part_ml[p];
#pragma unroll
                        for (int k = 0; k < V; k += 2)
                            *reinterpret_cast<float2 *>(&v[j][k]) =
                                *reinterpret_cast<const float2 *>(a.part_o + p * D + lane * V + k);
                    }
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    bad |= ml[j].y < 0.f;
                    if (ml[j].y == 0.f) continue;  // no part, or one without a key for this row
                    const float mn = fmaxf(M, ml[j].x), ref = mn == -INFINITY ? 0.f : mn;
                    const float f = mma::fast_exp2(M - ref), g = mma::fast_exp2(ml[j].x - ref);
                    M = mn;
                    L = fmaf(ml[j].y, g, L * f);
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = fmaf(v[j][k], g, acc[k] * f);
                }
            }
        if (W > 1) {
            __syncthreads();  // (the pass before has been read)
#pragma unroll
            for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = acc[k];
            if (lane == 0) {
                s_m[warp] = M;
                s_l[warp] = bad ? -1.f : L;
            }
            __syncthreads();
            if (!live || part) continue;
            M = -INFINITY;
            L = 0.f;
            bad = false;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                M = fmaxf(M, s_m[warp + w]);
                bad |= s_l[warp + w] < 0.f;
            }
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float f = mma::fast_exp2(s_m[warp + w] - ref);
                L = fmaf(s_l[warp + w], f, L);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] = fmaf(s_acc[warp + w][lane * V + k], f, acc[k]);
            }
        }
        if (!live) continue;
        const int row = row0 + r;
        const size_t at = (size_t)(row / a.G) * a.Hq + hk * a.G + row % a.G;
        const float inv = 1.f / L;
#pragma unroll
        for (int k = 0; k < V; k += 2)
            *reinterpret_cast<uint32_t *>(a.out + at * D + lane * V + k) =
                bad ? 0u : mma::pack_bf16(acc[k] * inv, acc[k + 1] * inv);
        if (lane == 0) a.lse[at] = bad ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    }
}

template <int D, int RW, int CW>
cudaError_t launch(const Attn &a, bool after_gate, cudaStream_t st) {
    CUtensorMap mk, mv;
    const long long rows = (long long)a.c.num_pages * a.c.Hkv * a.c.ps;
    const int box = a.c.ps < kTile ? a.c.ps : kTile;
    if (!make_tma_rows(&mk, a.k, rows, D, box) || !make_tma_rows(&mv, a.v, rows, D, box))
        return cudaErrorInvalidValue;
    const int bytes = (int)RowsSmem<D, CW>::kBytes;
    const cudaError_t rc = allow_smem<rows_kernel<D, RW, CW>>(bytes);
    if (rc != cudaSuccess) return rc;
    RowsArgs ra;
    ra.a = a;
    ra.psh = __builtin_ctz((unsigned)a.c.ps);
    ra.wait_limit = kDefaultWaitLimit;
    note_launches(1);
    if (after_gate)
        return launch_after(rows_kernel<D, RW, CW>, a.ctas, 32 * (CW + 1), bytes, st, mk, mv, ra);
    rows_kernel<D, RW, CW><<<a.ctas, 32 * (CW + 1), bytes, st>>>(mk, mv, ra);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const Attn &a, bool after_gate, cudaStream_t st) {
    return a.rows == 16   ? launch<D, 1, 4>(a, after_gate, st)
           : a.rows == 32 ? launch<D, 2, 4>(a, after_gate, st)
                          : launch<D, 4, 8>(a, after_gate, st);
}

}  // namespace

cudaError_t launch_rows(const Attn &a, bool after_gate, cudaStream_t st) {
    const cudaError_t rc = a.D == 64 ? launch_d<64>(a, after_gate, st) : launch_d<128>(a, after_gate, st);
    return rc == cudaSuccess ? launch_merge_runs(a, st) : rc;
}

cudaError_t launch_merge_runs(const Attn &a, cudaStream_t st) {
    const dim3 grid(a.ctas, (a.chunk ? kJobRows : a.rows) / merge_rows(a.chunk));
    note_launches(1);
    if (a.D == 64)
        return a.chunk ? launch_after(merge_runs_kernel<64, true>, grid, kMergeThreads, 0, st, a)
                       : launch_after(merge_runs_kernel<64, false>, grid, kMergeThreads, 0, st, a);
    return a.chunk ? launch_after(merge_runs_kernel<128, true>, grid, kMergeThreads, 0, st, a)
                   : launch_after(merge_runs_kernel<128, false>, grid, kMergeThreads, 0, st, a);
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
        a->c_open = static_cast<int *>(take(4 * (size_t)a->ctas));
        a->c_last = static_cast<int *>(take(4 * ents));
        a->part_ml = static_cast<float2 *>(take(sizeof(float2) * parts));
        a->part_o = static_cast<float *>(take(sizeof(float) * parts * a->D));
    }
    if (!a->dense && !a->chunk) {
        a->tiles = static_cast<int *>(take(4 * n));
        a->ublk = static_cast<int *>(take(4 * n * a->ucap));
        a->umask = static_cast<unsigned long long *>(take(8 * n * a->ucap));
    }
    if (a->chunk && a->dense) {
        a->own_off = static_cast<int *>(take(4 * ((size_t)a->c.num_seqs + 1)));
        a->unit_off = static_cast<long long *>(take(8 * ((size_t)a->w_cap + 1)));
    }
    if (a->chunk && !a->dense) {
        const size_t lists = (size_t)a->c.num_seqs * a->n_max * a->c.Hkv;
        const size_t slots = (size_t)a->c.total * a->Hq * (a->km1 + 1);
        a->counts = static_cast<int *>(take(4 * (lists + a->c.total)));
        a->tok = a->counts + lists;
        a->list_off = static_cast<int *>(take(4 * lists));
        a->used_off = static_cast<int *>(take(4 * ((size_t)a->c.num_seqs + 1)));
        a->jobs = static_cast<int2 *>(take(8 * (size_t)a->job_cap));
        a->halves = static_cast<int2 *>(take(8 * (size_t)a->job_cap));
        a->n_jobs = static_cast<int *>(take(12));
        a->list = static_cast<int *>(take(4 * (size_t)a->list_cap));
        a->sel = static_cast<int2 *>(take(8 * (size_t)a->c.total * a->Hq * a->km1));
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
    // (token, head of the group) and lists are 32-bit.  (us at 64 rows in this file's
    // kernel and 68 in the other, 32 / 8 heads of 128, caches of 32768: one sequence 59
    // and 60 with selection, 44 and 70 over all blocks; 8 sequences 217 and 192, 214 and
    // 193; 32 sequences 732 and 612, 777 and 698)
    const long long lists = a->dense ? 0 : (long long)a->c.num_seqs * n_max * a->c.Hkv;
    a->list_cap = (long long)a->c.total * Hq * a->km1;
    // From 33 rows on an entry's warps have four times 16 rows to multiply for every
    // key, which by then bounds them; so do many entries there, but for short blocks
    // (jobs of few tiles) and, over all blocks, heads of 64.  (us here and there, 36 to
    // 64 rows, caches of 16384, blocks of 512: 8 sequences of 8 kv heads 132 to 147 and
    // 124 to 127 with selection, 118 to 122 and 108 to 112 over all blocks, 99 to 109
    // and 89 to 92 with selection and heads of 64; 32 sequences 408 to 446 and 337 to
    // 363.  Against it: blocks of 128 137 and 152, heads of 64 over all blocks 89 and 95.
    // Blocks of 256 were not measured)
    const bool many = rows > 32 && (long long)a->c.num_seqs * a->c.Hkv >= 64 &&
                      (a->dense ? D == 128 : bs >= 512);
    a->chunk = (rows > kMaxRows || many) && (long long)a->c.total * a->G < (1ll << 26) &&
               lists < (1ll << 30) && a->list_cap < (1ll << 31);
    if (a->chunk) {
        const long long w0 = (long long)a->c.num_seqs * ((rows + kJobRows - 1) / kJobRows);
        const long long w1 = (long long)a->c.total * a->G / kJobRows + a->c.num_seqs;
        a->w_cap = (int)(w0 < w1 ? w0 : w1);
        a->job_cap = a->list_cap / kJobRows + (lists < a->list_cap ? lists : a->list_cap) + 1;
        if ((long long)a->w_cap * a->c.Hkv >= (1ll << 30) ||
            a->c.tile_slots(a->G, 128, 1) * a->c.Hkv >= (1ll << 31))
            return MOBA_ERR_UNSUPPORTED;
    }
    const long long ucap = (long long)a->rows * (a->km1 + 1);
    a->ucap = a->dense ? 0 : (int)(ucap < n_max ? ucap : n_max);
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
    cudaError_t e = a.chunk && !a.dense ? launch_chunk_gate(a, st) : launch_gate(a, st);
    const bool gated = !a.dense || a.idx;
    if (e == cudaSuccess && a.chunk) e = launch_plan(a, gated, st);
    if (e == cudaSuccess) e = a.chunk ? launch_chunk(a, st) : launch_rows(a, gated, st);
    if (own) {
        const cudaError_t f = cudaFreeAsync(own, st);
        if (e == cudaSuccess) e = f;
    }
    return cuda_result(e);
}
