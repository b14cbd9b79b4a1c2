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
//   1. The plan (one CTA) checks the groups and makes spans: a tile of rows with a range of
//      keys.  A group's rows lie one behind the other, whatever sequences they are of, so
//      that its tiles see the prefix whole, without a mask; what is behind the prefix is
//      each sequence's own.
//   2. Big spans, 256 rows, are jobs of the tcgen05 kernel of long chunks: groups of more
//      rows than a small span holds, and the own keys in calls of many new tokens.
//   3. Small spans, 16 rows, are streamed on mma.sync: a decode step's own keys, and the
//      prefixes of groups that fit.
//   4. Every part of 2 and 3 leaves partial sums, which the merge joins.
#include "moba_mma.cuh"
#include "moba_paged_attn.cuh"
#include "moba_ptx.cuh"

namespace moba {
namespace paged {
namespace {

constexpr int kSmallRows = 16;   // of a small span
constexpr int kUnit = 16;        // keys that a warp takes at a time: never more than a page
constexpr int kBigKeys = 128;    // of a key tile of the tcgen05 kernel
constexpr int kStreamWarps = 4, kStreamCtas = 3;  // of a CTA, of an SM
constexpr int kMinUnits = 6;     // units of a warp's run at least, where there are few
// The start of a span on a kv head counts as that many units, its rows and sums being
// what they cost: runs of equal units then take equal time.
constexpr int kSmallStart = 2;
// From kDynamic units a warp on, a quarter of them is cut into runs (kShort a warp) that the
// warps take as they become free: SMs differ, by their distance from the memory, in what
// they get through (160 K to 210 K cycles of equal runs).
constexpr int kDynamic = 24, kShort = 2;

struct SharedArgs {
    Attn a;
    const int *cu_groups;        // [n_groups + 1]
    const int *prefix_lens;      // [n_groups]
    int n_groups;
    int small_rows;              // groups of up to that many rows are small spans
    int cap_big, cap_small;      // spans at most
    int own_cap;                 // of them sequences' own
    int warps;                   // of the streaming kernel
    int psh;                     // log2(page size)
    // scratch
    Span *tiles_small;           // [cap_small]
    long long *off_small;        // [cap_small + 1] units before each, times the kv heads
    int *rep;                    // [n_groups] the sequence whose pages are read (num_seqs: none, -1: a wrong group)
    int *at;                     // [n_groups] its first span << 1 | big, or -1
    int4 *info;                  // [num_seqs] tokens shared, the group's first row, its first span, big
    int *small_first, *small_last;  // [cap_small * Hkv] the runs that the span on the kv head lies in
    float *small_o;              // [cap_small * Hkv + runs][kSmallRows][D] partial sums, as part_o
    float2 *small_ml;            // [cap_small * Hkv + runs][kSmallRows]
};

// ----------------------------------------------------------------------------
// plan
// ----------------------------------------------------------------------------
constexpr int kHeld = 1024;      // sequences and groups whose tables fit shared memory

// inclusive sums over the CTA's T threads, N at a time
template <int T, int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long (*warps)[32], long long (&total)[N]) {
    constexpr int W = T / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, v[i], o);
            if (lane >= o) v[i] += y;
        }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (lane == 31) warps[i][warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        long long s = lane < W ? warps[i][lane] : 0;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        total[i] = __shfl_sync(0xffffffffu, s, W - 1);
        const long long before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
        v[i] += warp > 0 ? before : 0;
    }
}

// T threads.  HELD: as many sequences and groups as shared memory has room for, so that
// the searches cost little.
template <int T, bool HELD>
__global__ void __launch_bounds__(T) plan_spans_kernel(SharedArgs x) {
    __shared__ long long warps[4][32];
    __shared__ int s_cu[HELD ? kHeld + 1 : 1], s_len[HELD ? kHeld : 1], s_grp[HELD ? kHeld + 1 : 1];
    __shared__ int s_pre[HELD ? kHeld : 1], s_rep[HELD ? kHeld : 1], s_at[HELD ? kHeld : 1];
    const Attn &a = x.a;
    const Cache &c = a.c;
    let_next();
    after_previous();
    const int tid = threadIdx.x, ns = c.num_seqs, ng = x.n_groups, G = a.G, Hkv = c.Hkv;
    if (HELD) {
        for (int i = tid; i <= ns; i += T) {
            s_cu[i] = __ldg(c.cu + i);
            if (i < ns) s_len[i] = __ldg(c.lens + i);
        }
        for (int i = tid; ng > 0 && i <= ng; i += T) {
            s_grp[i] = __ldg(x.cu_groups + i);
            if (i < ng) s_pre[i] = __ldg(x.prefix_lens + i);
        }
        __syncthreads();
    }
    auto cu = [&](int i) { return HELD ? s_cu[i] : __ldg(c.cu + i); };
    auto grp = [&](int i) { return HELD ? s_grp[i] : __ldg(x.cu_groups + i); };
    auto pre = [&](int i) { return HELD ? s_pre[i] : __ldg(x.prefix_lens + i); };
    int *rep = HELD ? s_rep : x.rep, *at = HELD ? s_at : x.at;
    auto sync = [&] {
        if (!HELD) __threadfence_block();
        __syncthreads();
    };
    auto seq = [&](int b, Seq &s) { return c.check(cu(b), cu(b + 1), HELD ? s_len[b] : __ldg(c.lens + b), s); };
    // groups: offsets that lead nowhere void all of them
    bool wrong = false;
    for (int g = tid; ng > 0 && g <= ng; g += T) {
        const int p = grp(g);
        wrong |= p < 0 || p > ns || (g > 0 && grp(g - 1) > p);
    }
    const bool none = __syncthreads_or(wrong) || ng == 0;
    for (int g = tid; g < ng; g += T) {
        const int p = pre(g);
        const bool ok = !none && p >= 0 && p % c.ps == 0 && p <= (long long)c.max_pages * c.ps;
        rep[g] = ok ? ns : -1;
    }
    sync();
    // the group of sequence b, or -1
    auto group_of = [&](int b) {
        if (none) return -1;
        int g = 0, hi = ng - 1;
        while (g < hi) {
            const int mid = (g + hi + 1) >> 1;
            if (grp(mid) <= b) g = mid; else hi = mid - 1;
        }
        return grp(g) <= b && b < grp(g + 1) ? g : -1;
    };
    // every sequence's say: the first with new tokens lends its pages; one that is refused,
    // or has new tokens inside the prefix, voids the group
    for (int b0 = 0; b0 < ns; b0 += T) {
        const int b = b0 + tid;
        Seq s;
        const int state = b < ns ? seq(b, s) : (int)kSeqEmpty;
        if (state != kSeqEmpty) {
            const int g = group_of(b);
            if (g >= 0) atomicMin(rep + g, state == kSeqOk && pre(g) <= s.len - s.n ? b : -1);
        }
        if (state == kSeqBad) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        if (__syncthreads_or(state == kSeqBad))
            for (int r = b0; r < min(b0 + T, ns); ++r) {
                Seq y;
                if (seq(r, y) == kSeqBad) clear_refused(a, y, 0, a.Hq, tid, T);
            }
    }
    sync();
    // the groups' spans
    long long nb = 0, ub = 0, nm = 0, um = 0;  // big and small ones so far, and their units
    for (int g0 = 0; g0 < ng; g0 += T) {
        const int g = g0 + tid;
        long long v[4] = {0, 0, 0, 0}, total[4];
        int row0 = 0, rows = 0, p = 0, n = 0, lender = -1;
        bool big = false;
        if (g < ng) {
            lender = HELD ? rep[g] : __ldcg(rep + g);  // (where the atomics left it)
            if (lender < 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
            p = pre(g);
            if (lender >= 0 && lender < ns && p > 0) {
                row0 = cu(grp(g)) * G;
                rows = cu(grp(g + 1)) * G - row0;
                big = rows > x.small_rows;
                n = big ? (rows + kJobRows - 1) / kJobRows : 1;
                v[big ? 0 : 2] = n;
                v[big ? 1 : 3] = (long long)n * Hkv * (big ? (p + kBigKeys - 1) / kBigKeys + kBigStart
                                                           : (p + kUnit - 1) / kUnit + kSmallStart);
            }
        }
        const long long mine_n = v[0] + v[2], mine_u = v[1] + v[3];
        block_scan<T>(v, warps, total);
        if (g < ng) {
            const long long i0 = (big ? nb + v[0] : nm + v[2]) - mine_n, u0 = (big ? ub + v[1] : um + v[3]) - mine_u;
            const int cap = big ? x.cap_big : x.cap_small;
            Span *tiles = big ? a.tiles_big : x.tiles_small;
            long long *off = big ? a.off_big : x.off_small;
            for (int i = 0; i < n && i0 + i < cap; ++i) {
                Span t;
                t.row0 = row0 + i * kJobRows;
                t.nrows = min(rows - i * kJobRows, kJobRows);
                t.b = lender;
                t.full = 1;
                t.key0 = 0;
                t.key_end = p;
                t.pdelta = t.pad = 0;
                tiles[i0 + i] = t;
                off[i0 + i + 1] = u0 + mine_u / n * (i + 1);
            }
            // (more than there is room for: from offsets that overlap)
            at[g] = n > 0 && i0 + n <= cap ? (int)i0 << 1 | big : -1;
        }
        nb += total[0];
        ub += total[1];
        nm += total[2];
        um += total[3];
    }
    sync();
    const int groups_spans[2] = {(int)min(nb, (long long)x.cap_big), (int)min(nm, (long long)x.cap_small)};
    // the sequences' own
    const int cap = a.chunk ? x.cap_big : x.cap_small, tile_rows = a.chunk ? kJobRows : kSmallRows;
    const int unit = a.chunk ? kBigKeys : kUnit, start = a.chunk ? kBigStart : kSmallStart;
    Span *tiles = a.chunk ? a.tiles_big : x.tiles_small;
    long long *off = a.chunk ? a.off_big : x.off_small;
    long long &nt = a.chunk ? nb : nm, &ut = a.chunk ? ub : um;
    for (int b0 = 0; b0 < ns; b0 += T) {
        const int b = b0 + tid;
        long long v[2] = {0, 0}, total[2];
        Seq s;
        int first = 0, rows = 0, pdelta = 0;
        int4 info = make_int4(0, 0, 0, 0);
        if (b < ns && seq(b, s) == kSeqOk) {
            const int g = group_of(b), t = g >= 0 ? at[g] : -1;
            if (t >= 0) {
                first = pre(g);
                info = make_int4(first, cu(grp(g)) * G, t >> 1, t & 1);
            }
            rows = s.n * G;
            pdelta = s.len - s.n - s.row0;
            v[0] = (rows + tile_rows - 1) / tile_rows;
            for (int r = 0; r < rows; r += tile_rows)
                v[1] += (s.len - s.n + (min(r + tile_rows, rows) - 1) / G - first) / unit + 1 + start;
            v[1] *= Hkv;
        }
        const long long mine_n = v[0], mine_u = v[1];
        block_scan<T>(v, warps, total);
        if (b < ns) {
            long long i = nt + v[0] - mine_n, u = ut + v[1] - mine_u;
            x.info[b] = info;
            for (int r = 0; r < rows && i < cap; r += tile_rows, ++i) {
                Span t;
                t.row0 = s.row0 * G + r;
                t.nrows = min(rows - r, tile_rows);
                t.b = b;
                t.full = 0;
                t.key0 = first;
                t.key_end = (t.row0 + t.nrows - 1) / G + pdelta + 1;
                t.pdelta = pdelta;
                t.pad = 0;
                tiles[i] = t;
                u += (long long)Hkv * ((t.key_end - first + unit - 1) / unit + start);
                off[i + 1] = u;
            }
        }
        nt += total[0];
        ut += total[1];
    }
    if (tid == 0) {
        // spans, and those of groups among them
        *reinterpret_cast<int4 *>(a.n_spans) = make_int4((int)min(nb, (long long)x.cap_big), (int)min(nm, (long long)x.cap_small),
                                                         groups_spans[0], groups_spans[1]);
        a.n_spans[4] = 0;
        a.off_big[0] = x.off_small[0] = 0;
    }
}

// ----------------------------------------------------------------------------
// small spans
// ----------------------------------------------------------------------------
// The units (16 keys of a span on a kv head) of all spans form one sequence that is cut
// into runs, one per warp.  A warp works alone: it brings K and V (boxes of 16 keys) into
// a ring of its own and there is no barrier among warps; a span that ends costs its
// partial sums and no more, and the copies run ahead over it.  A lane takes K and V from
// the ring 16 bytes at a time, straight into the registers of its fragments.  For that
// the products take their dimensions in an order of their own: of 64 dimensions, a lane's
// 16 neighbours are its pairs of four steps of q k, and 8 neighbours one column of each of
// eight steps of p v, whose pairs are two keys' values.
// Bound: HBM.  16 rows with 16384 keys on 32 kv heads and 16 times up to 2000 more, 541 MB:
// 88 us, 6.15 TB/s, 0.91 of the copy rate.  (By cp.async, 16 bytes a lane in requests of 64
// bytes, it took 105 us, whatever the warps and stages.)
template <int D>
struct Ring {
    static constexpr int C = D / 32, O = D / 64;
    static constexpr int kBox = kUnit * 128;       // 64 dimensions of the keys, 128-byte swizzle
    static constexpr int kStage = 2 * O * kBox;    // K, then V
    static constexpr int kStages = 2 * 128 / D;
    static constexpr int kBytes = kStreamWarps * kStages * kStage + 1024;
};

template <int D>
__global__ void __launch_bounds__(32 * kStreamWarps, kStreamCtas)
    stream_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                  const __grid_constant__ SharedArgs x) {
    using mma::fast_exp2;
    using mma::mma16816;
    using mma::pack_bf16;
    using R = Ring<D>;
    constexpr int C = R::C, O = R::O, ST = R::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ __align__(8) unsigned long long s_bar[kStreamWarps][ST];
    __shared__ int s_abort;
    const Attn &a = x.a;
    const Cache &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n8 = lane >> 2, c4 = lane & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStreamWarps; ++i)
            for (int s = 0; s < ST; ++s) ptx::mbar_init(ptx::saddr(&s_bar[i][s]), 1);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    after_previous();
    let_next();
    ptx::Ctl ctl{&s_abort, a.status, kDefaultWaitLimit};
    const uint32_t raw = ptx::saddr(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t ring = base + warp * ST * R::kStage, bars = ptx::saddr(&s_bar[warp][0]);
    const uint8_t *mine = smem_raw + (ring - raw);
    const int gw = blockIdx.x * kStreamWarps + warp, G = a.G, Hkv = c.Hkv, ps = c.ps;
    const int spans = a.n_spans[1];
    const long long total = x.off_small[spans], most = (total + kMinUnits - 1) / kMinUnits;
    const bool dynamic = total > (long long)x.warps * kDynamic;
    const long long even = dynamic ? total - total / 4 : total;  // units of the runs that are one for each warp
    const int runs = dynamic ? x.warps * (1 + kShort) : (int)(most < x.warps ? most : x.warps);
    int issued = 0, used = 0;  // stages so far
    for (int run = gw, next = 0; run < runs; run = next) {
        if (dynamic && lane == 0) next = atomicAdd(a.n_spans + 4, 1);
        const long long firsts = dynamic ? x.warps : runs;
        auto begin = [&](int r) {
            return r <= firsts ? even * r / firsts : even + (total - even) * (r - firsts) / (x.warps * kShort);
        };
        const long long u0 = begin(run);
        const int n = (int)(begin(run + 1) - u0);
        int w = 0;  // the span with unit u0: the last that starts at or before it
        for (int k = spans; k > 1;) {
            const int step = (k + 31) / 32;
            const bool below = lane * step < k && x.off_small[w + lane * step] <= u0;
            const int last = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
            k = min(step, k - last * step);
            w += last * step;
        }
        // ---- copies ----
        int ahead = 0, wa = w;              // units of the run that have been issued; a span at or before the next
        int place = 0;                      // lane: its unit of the 32 at hand: first row of the pools (-1: no keys)
        unsigned long long bad_units = 0;   // of the last 64 units
        auto look_up = [&] {
            int wl = wa;
            bool bad = false;
            place = -1;
            if (ahead + lane < n) {
                const long long u = u0 + ahead + lane;
                while (x.off_small[wl + 1] <= u) ++wl;
                const Span s = x.tiles_small[wl];
                const long long o = x.off_small[wl], T = (x.off_small[wl + 1] - o) / Hkv;
                const int hk = (int)((u - o) / T), i = (int)(u - o - hk * T) - kSmallStart;
                if (i >= 0) {
                    const int key = s.key0 + i * kUnit;
                    const int page = __ldg(c.table + (size_t)s.b * c.max_pages + (key >> x.psh));
                    bad = (unsigned)page >= (unsigned)c.num_pages;
                    // (some memory of the pool for a page outside it: its rows are dropped)
                    place = (((bad ? 0 : page) * Hkv + hk) << x.psh) + (key & (ps - 1));
                }
            }
            const unsigned long long ballot = __ballot_sync(0xffffffffu, bad);
            const int at = ahead & 63;
            bad_units = (bad_units & ~(0xffffffffull << at)) | ballot << at;
            wa = __shfl_sync(0xffffffffu, wl, min(31, n - 1 - ahead));
        };
        auto issue = [&] {
            if (ahead >= n) return;
            if ((ahead & 31) == 0) look_up();
            const int at = __shfl_sync(0xffffffffu, place, ahead & 31);
            ++ahead;
            if (at < 0) return;
            if (lane == 0) {
                const uint32_t bar = bars + 8 * (issued % ST), dst = ring + (issued % ST) * R::kStage;
                ptx::mbar_expect_tx(bar, R::kStage);
#pragma unroll
                for (int v = 0; v < 2; ++v)
#pragma unroll
                    for (int q = 0; q < O; ++q)
                        asm volatile(
                            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                            "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst + (v * O + q) * R::kBox),
                            "l"(reinterpret_cast<uint64_t>(v ? &tmap_v : &tmap_k)), "r"(bar), "r"(q * 64), "r"(at)
                            : "memory");
            }
            ++issued;
        };
#pragma unroll 1
        for (int i = 0; i < ST - 1; ++i) issue();
        bool ok = true;
        // ---- parts: the run's units of one span on one kv head ----
        for (int j = 0; ok && j < n;) {
            while (x.off_small[w + 1] <= u0 + j) ++w;
            const Span s = x.tiles_small[w];
            const long long in = u0 + j - x.off_small[w], T = (x.off_small[w + 1] - x.off_small[w]) / Hkv;
            const int hk = (int)(in / T), v0 = (int)(in - hk * T), cnt = (int)min(T - v0, (long long)(n - j));
            const int e = w * Hkv + hk;
            // this lane's rows, n8 and n8 + 8
            int see[2];
            uint4 qr[C][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = n8 + 8 * h, row = s.row0 + r, t = row / G;
                const bool live = r < s.nrows;
                // last key that the row sees (no row: whatever, its scores do not matter)
                see[h] = live && !s.full ? t + s.pdelta : 0x7fffffff;
                const __nv_bfloat16 *src = a.q + ((size_t)t * a.Hq + hk * G + (row - t * G)) * D + 16 * c4;
#pragma unroll
                for (int i = 0; i < C; ++i)
                    qr[i][h] = live ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * (i >> 1) + 8 * (i & 1)))
                                    : make_uint4(0, 0, 0, 0);
            }
            float o[O][8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < O; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k)
#pragma unroll
                    for (int z = 0; z < 4; ++z) o[i][k][z] = 0.f;
            bool bad = false;
            for (int v = v0; v < v0 + cnt; ++v, ++j) {
                issue();
                if (v < kSmallStart) continue;  // (units that stand for the span's start)
                ok = __all_sync(0xffffffffu, ptx::wait_fast(bars + 8 * (used % ST), (used / ST) & 1, ctl));
                if (!ok) break;
                bad |= bad_units >> (j & 63) & 1;
                const int key0 = s.key0 + (v - kSmallStart) * kUnit, nv = s.key_end - key0;
                const uint8_t *stage = mine + (used % ST) * R::kStage;
                ++used;
                // 16 bytes of row r of a box (r & 7 as in the address of its swizzle)
                auto piece = [&](int box, int r, int p) {
                    return *reinterpret_cast<const uint4 *>(stage + box * R::kBox + r * 128 + ((p ^ (r & 7)) << 4));
                };
                float sc[2][4];
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[z][k] = 0.f;
#pragma unroll
                for (int q = 0; q < C; ++q) {
                    const uint32_t lo[4] = {qr[q][0].x, qr[q][1].x, qr[q][0].y, qr[q][1].y};
                    const uint32_t hi[4] = {qr[q][0].z, qr[q][1].z, qr[q][0].w, qr[q][1].w};
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const uint4 k = piece(q >> 1, n8 + 8 * z, 2 * c4 + (q & 1));
                        mma16816(sc[z], lo, k.x, k.y);
                        mma16816(sc[z], hi, k.z, k.w);
                    }
                }
                float mx[2] = {-INFINITY, -INFINITY}, mu[2];
                const bool open = key0 + kUnit - 1 <= min(see[0], see[1]) && nv >= kUnit;
                if (__all_sync(0xffffffffu, open)) {
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int k = 0; k < 4; ++k) mx[k >> 1] = fmaxf(mx[k >> 1], sc[z][k]);
                } else {
#pragma unroll
                    for (int z = 0; z < 2; ++z)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int key = z * 8 + 2 * c4 + (k & 1);
                            if (key >= nv || key0 + key > see[k >> 1]) sc[z][k] = -INFINITY;
                            mx[k >> 1] = fmaxf(mx[k >> 1], sc[z][k]);
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
                        for (int q = 0; q < O; ++q)
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                o[q][k][2 * h] *= r;
                                o[q][k][2 * h + 1] *= r;
                            }
                    }
                }
                mu[0] = m[0] == -INFINITY ? 0.f : m[0];
                mu[1] = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sc[z][k] = fast_exp2(fmaf(sc[z][k], a.scale_log2, -mu[k >> 1]));
                        l[k >> 1] += sc[z][k];
                    }
                const uint32_t pa[4] = {pack_bf16(sc[0][0], sc[0][1]), pack_bf16(sc[0][2], sc[0][3]),
                                        pack_bf16(sc[1][0], sc[1][1]), pack_bf16(sc[1][2], sc[1][3])};
#pragma unroll
                for (int q = 0; q < O; ++q) {
                    uint4 p[4];  // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = 2 * c4 + (k & 1) + 8 * (k >> 1);
                        p[k] = piece(O + q, r, n8);
                        // (keys that no row sees may never have been written: zeros)
                        if (r >= nv) p[k] = make_uint4(0, 0, 0, 0);
                    }
                    const uint32_t x0[4] = {p[0].x, p[0].y, p[0].z, p[0].w}, x1[4] = {p[1].x, p[1].y, p[1].z, p[1].w},
                                   x8[4] = {p[2].x, p[2].y, p[2].z, p[2].w}, x9[4] = {p[3].x, p[3].y, p[3].z, p[3].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma16816(o[q][2 * k], pa, __byte_perm(x0[k], x1[k], 0x5410), __byte_perm(x8[k], x9[k], 0x5410));
                        mma16816(o[q][2 * k + 1], pa, __byte_perm(x0[k], x1[k], 0x7632), __byte_perm(x8[k], x9[k], 0x7632));
                    }
                }
                __syncwarp();  // (the stage has been read: the next copy may go there)
            }
            // ---- the part's sums ----
            if (!ok) break;
            if (v0 + cnt <= kSmallStart) continue;  // (it had no keys)
            if (bad && lane == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
            if (lane == 0) {
                if (v0 <= kSmallStart) x.small_first[e] = run;
                if (v0 + cnt == T) x.small_last[e] = run;
            }
            const size_t slot = ((size_t)e + run) * kSmallRows;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
                l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
                const int r = n8 + 8 * h;
                if (r >= s.nrows) continue;
                float *dst = x.small_o + (slot + r) * D + 16 * c4;
#pragma unroll
                for (int q = 0; q < O; ++q)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int z = 0; z < 8; z += 4)
                            *reinterpret_cast<float4 *>(dst + 64 * q + 8 * k + z) =
                                make_float4(o[q][z][2 * h + k], o[q][z + 1][2 * h + k], o[q][z + 2][2 * h + k],
                                            o[q][z + 3][2 * h + k]);
                if (c4 == 0) x.small_ml[slot + r] = make_float2(m[h], bad ? -1.f : l[h]);
            }
        }
        if (!ok) {  // copies in flight land before the CTA ends
            for (; used < issued; ++used) ptx::drain_bar(bars + 8 * (used % ST), (used / ST) & 1, kDefaultWaitLimit);
            return;
        }
        next = dynamic ? x.warps + __shfl_sync(0xffffffffu, next, 0) : runs;
    }
}

// ----------------------------------------------------------------------------
// merge
// ----------------------------------------------------------------------------
// A CTA takes up to kMergeRows rows of a sequence's own span on a kv head, whose parts and
// whose group's it looks up once; W warps to a row, every W-th part each, where rows are
// few (they have many parts then).
constexpr int kMergeWarps = 8, kMergeRows = 32;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps, 4) merge_spans_kernel(SharedArgs x) {
    constexpr int V = D / 32, U = 4;
    __shared__ float s_acc[kMergeWarps][D], s_m[kMergeWarps], s_l[kMergeWarps];
    const Attn &a = x.a;
    after_previous();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.G, Hkv = a.c.Hkv;
    const bool chunk = a.chunk;
    const int4 n = *reinterpret_cast<const int4 *>(a.n_spans);
    const int w = (int)blockIdx.x / Hkv + (chunk ? n.z : n.w), hk = blockIdx.x % Hkv;
    if (w >= (chunk ? n.x : n.y)) return;
    const Span s = (chunk ? a.tiles_big : x.tiles_small)[w];
    const int r0 = blockIdx.y * kMergeRows, rows = min(s.nrows - r0, kMergeRows);
    if (rows <= 0) return;
    const int4 info = x.info[s.b];
    const int W = rows > 4 ? 1 : rows > 2 ? 2 : rows > 1 ? 4 : 8, part = warp % W;
    for (int ri = warp / W; ri < (W > 1 ? kMergeWarps / W : rows); ri += kMergeWarps / W) {
        const bool live = ri < rows;
        const int row = s.row0 + r0 + ri;
        float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        bool bad = false;
        // the parts of row r of span e / Hkv on kv head e % Hkv
        auto add = [&](bool big, int e, int r) {
            const int slots = big ? kJobRows : kSmallRows;
            const int c0 = max((big ? a.c_first : x.small_first)[e], 0);
            const int c1 = min((big ? a.c_last : x.small_last)[e], (big ? a.ctas : x.warps * (1 + kShort)) - 1);
            const float *o = big ? a.part_o : x.small_o;
            const float2 *ml = big ? a.part_ml : x.small_ml;
            for (int c = c0 + part; c <= c1; c += W * U) {
                float2 z[U];
                float v[U][V];
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    z[j] = make_float2(-INFINITY, 0.f);
                    if (c + W * j <= c1) {
                        const size_t p = ((size_t)e + c + W * j) * slots + r;
                        z[j] = ml[p];
#pragma unroll
                        for (int k = 0; k < V; k += 2)
                            *reinterpret_cast<float2 *>(&v[j][k]) =
                                *reinterpret_cast<const float2 *>(o + p * D + lane * V + k);
                    }
                }
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    bad |= z[j].y < 0.f;
                    if (z[j].y == 0.f) continue;  // no part, or one without a key for this row
                    const float mn = fmaxf(M, z[j].x), ref = mn == -INFINITY ? 0.f : mn;
                    const float f = mma::fast_exp2(M - ref), g = mma::fast_exp2(z[j].x - ref);
                    M = mn;
                    L = fmaf(z[j].y, g, L * f);
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[k] = fmaf(v[j][k], g, acc[k] * f);
                }
            }
        };
        if (live) {
            if (info.x > 0) {
                const int at = row - info.y, tile = info.w ? kJobRows : kSmallRows;
                add(info.w != 0, (info.z + at / tile) * Hkv + hk, at % tile);
            }
            add(chunk, w * Hkv + hk, r0 + ri);
        }
        if (W > 1) {  // (one round: every warp is here)
#pragma unroll
            for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = acc[k];
            if (lane == 0) {
                s_m[warp] = M;
                s_l[warp] = bad ? -1.f : L;
            }
            __syncthreads();
            if (!live || part) return;
            M = -INFINITY;
            L = 0.f;
            bad = false;
            for (int i = warp; i < warp + W; ++i) {
                M = fmaxf(M, s_m[i]);
                bad |= s_l[i] < 0.f;
            }
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
            for (int i = warp; i < warp + W; ++i) {
                const float f = mma::fast_exp2(s_m[i] - ref);
                L = fmaf(s_l[i], f, L);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] = fmaf(s_acc[i][lane * V + k], f, acc[k]);
            }
        }
        const int t = row / G;
        const size_t at = (size_t)t * a.Hq + hk * G + (row - t * G);
        const float inv = 1.f / L;
#pragma unroll
        for (int k = 0; k < V; k += 2)
            *reinterpret_cast<uint32_t *>(a.out + at * D + lane * V + k) =
                bad ? 0u : mma::pack_bf16(acc[k] * inv, acc[k + 1] * inv);
        if (lane == 0) a.lse[at] = bad ? -INFINITY : (M + log2f(L)) * 0.69314718055994530942f;
    }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
size_t scratch(SharedArgs *x, void *base) {
    size_t off = 0;
    auto take = [&](size_t bytes) -> void * {
        void *p = base ? static_cast<char *>(base) + off : nullptr;
        off = (off + bytes + 255) & ~size_t(255);
        return p;
    };
    Attn &a = x->a;
    const size_t ns = a.c.num_seqs, ng = x->n_groups, nb = x->cap_big, nm = x->cap_small;
    a.n_spans = static_cast<int *>(take(32));
    a.tiles_big = static_cast<Span *>(take(sizeof(Span) * nb));
    a.off_big = static_cast<long long *>(take(8 * (nb + 1)));
    x->tiles_small = static_cast<Span *>(take(sizeof(Span) * nm));
    x->off_small = static_cast<long long *>(take(8 * (nm + 1)));
    x->rep = static_cast<int *>(take(4 * ng));
    x->at = static_cast<int *>(take(4 * ng));
    x->info = static_cast<int4 *>(take(sizeof(int4) * ns));
    a.c_first = static_cast<int *>(take(4 * nb * a.c.Hkv));
    a.c_last = static_cast<int *>(take(4 * nb * a.c.Hkv));
    x->small_first = static_cast<int *>(take(4 * nm * a.c.Hkv));
    x->small_last = static_cast<int *>(take(4 * nm * a.c.Hkv));
    const size_t big = nb ? (nb * a.c.Hkv + a.ctas) * kJobRows : 0;
    a.part_ml = static_cast<float2 *>(take(sizeof(float2) * big));
    a.part_o = static_cast<float *>(take(sizeof(float) * big * a.D));
    const size_t small = nm ? (nm * a.c.Hkv + (size_t)x->warps * (1 + kShort)) * kSmallRows : 0;
    x->small_ml = static_cast<float2 *>(take(sizeof(float2) * small));
    x->small_o = static_cast<float *>(take(sizeof(float) * small * a.D));
    return off;
}

// Sizes of a call whose cache has been checked (x->a.c is filled).
int make_shared(SharedArgs *x, int Hq, int D, int n_groups) {
    Attn &a = x->a;
    if (n_groups < 0) return MOBA_ERR_INVALID_ARG;
    if (n_groups > 65535) return MOBA_ERR_UNSUPPORTED;
    const int rc = make_attn(&a, Hq, D, 1 << 30);
    if (rc != MOBA_OK) return rc;
    const long long rows = (long long)a.c.total * a.G;
    if (rows >= (1ll << 26)) return MOBA_ERR_UNSUPPORTED;
    x->n_groups = n_groups;
    x->warps = sm_count() * kStreamCtas * kStreamWarps;
    x->psh = __builtin_ctz((unsigned)a.c.ps);
    x->small_rows = a.chunk ? 0 : kSmallRows;
    // sequences and groups with rows: each may leave a tile that is not full
    const long long seqs = a.c.num_seqs < a.c.total ? a.c.num_seqs : a.c.total;
    const long long groups = n_groups < seqs ? n_groups : seqs;
    const long long own = rows / (a.chunk ? kJobRows : kSmallRows) + seqs;
    const long long big = groups && rows > x->small_rows ? rows / kJobRows + groups : 0;
    const long long nb = big + (a.chunk ? own : 0), nm = a.chunk ? 0 : own + groups;
    if (nb * a.c.Hkv >= (1ll << 30) || nm * a.c.Hkv >= (1ll << 30)) return MOBA_ERR_UNSUPPORTED;
    x->own_cap = (int)own;
    x->cap_big = (int)nb;
    x->cap_small = (int)nm;
    return MOBA_OK;
}

cudaError_t launch_plan(const SharedArgs &x, cudaStream_t st) {
    note_launches(1);
    const int most = x.a.c.num_seqs > x.n_groups ? x.a.c.num_seqs : x.n_groups;
    if (most <= 128) plan_spans_kernel<128, true><<<1, 128, 0, st>>>(x);
    else if (most <= kHeld) plan_spans_kernel<1024, true><<<1, 1024, 0, st>>>(x);
    else plan_spans_kernel<1024, false><<<1, 1024, 0, st>>>(x);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_small(const SharedArgs &x, cudaStream_t st) {
    CUtensorMap mk, mv;
    const long long rows = (long long)x.a.c.num_pages * x.a.c.Hkv * x.a.c.ps;
    if (!make_tma_rows(&mk, x.a.k, rows, D, kUnit) || !make_tma_rows(&mv, x.a.v, rows, D, kUnit))
        return cudaErrorInvalidValue;
    const cudaError_t rc = allow_smem<stream_kernel<D>>(Ring<D>::kBytes);
    if (rc != cudaSuccess) return rc;
    note_launches(1);
    return launch_after(stream_kernel<D>, dim3(x.warps / kStreamWarps), dim3(32 * kStreamWarps), Ring<D>::kBytes, st, mk,
                        mv, x);
}

template <int D>
cudaError_t launch_merge(const SharedArgs &x, cudaStream_t st) {
    note_launches(1);
    return launch_after(merge_spans_kernel<D>, dim3((unsigned)(x.own_cap * x.a.c.Hkv), x.a.chunk ? kJobRows / kMergeRows : 1),
                        dim3(32 * kMergeWarps), 0, st, x);
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
    SharedArgs x = {};
    // any non-null, aligned addresses: only the sizes matter here
    const void *some = reinterpret_cast<const void *>(256);
    const int32_t *ints = static_cast<const int32_t *>(some);
    if (make_cache(&x.a.c, some, some, nullptr, ints, ints, ints, num_seqs, total, max_new, Hkv, D, 1, page_size,
                   max_pages, any_block(page_size)) != MOBA_OK ||
        make_shared(&x, Hq, D, n_groups) != MOBA_OK)
        return 0;
    return scratch(&x, nullptr);
}

MOBA_EXPORT int moba_paged_attn_shared(const void *q, const void *k_pages, const void *v_pages,
                                       const int32_t *page_table, const int32_t *cu_new, const int32_t *cache_lens,
                                       const int32_t *cu_groups, const int32_t *prefix_lens, void *out, float *lse,
                                       int num_seqs, int n_groups, int total, int max_new, int Hq, int Hkv, int D,
                                       int num_pages, int page_size, int max_pages, void *workspace,
                                       size_t workspace_bytes, void *stream) {
    if (!q || !out || !lse || (n_groups > 0 && (!cu_groups || !prefix_lens))) return MOBA_ERR_INVALID_ARG;
    SharedArgs x = {};
    Attn &a = x.a;
    int rc = make_cache(&a.c, k_pages, v_pages, nullptr, page_table, cu_new, cache_lens, num_seqs, total, max_new,
                        Hkv, D, num_pages, page_size, max_pages, any_block(page_size));
    if (rc == MOBA_OK) rc = make_shared(&x, Hq, D, n_groups);
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
    x.cu_groups = cu_groups;
    x.prefix_lens = prefix_lens;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const size_t need = scratch(&x, nullptr);
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
    scratch(&x, workspace);
    cudaError_t e = launch_plan(x, st);
    if (e == cudaSuccess && x.cap_big) e = launch_chunk_spans(a, st);
    if (e == cudaSuccess && x.cap_small) e = D == 64 ? launch_small<64>(x, st) : launch_small<128>(x, st);
    if (e == cudaSuccess) e = D == 64 ? launch_merge<64>(x, st) : launch_merge<128>(x, st);
    if (own) {
        const cudaError_t f = cudaFreeAsync(own, st);
        if (e == cudaSuccess) e = f;
    }
    return cuda_result(e);
}
