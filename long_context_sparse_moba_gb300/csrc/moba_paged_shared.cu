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
//      prefixes of groups that fit, or of all groups where they are short.
//   4. Every part of 2 and 3 leaves partial sums, which the merge joins.
// P is rounded to bf16 for the second product, as in the other attention kernels: relative
// to 64 bits outputs err by 0.0020 to 0.0024, of which the result's own rounding is 0.0016.  (In
// two bf16 pieces it would need that product twice, which bounds the chunks; a weight errs by 2^-8
// of itself at most, as does the result.)
// Measured (heads of 128 unless said): 64 forks of 32768 tokens with up to 512 of their own,
// 32 / 8 heads, 69 us (plan 3, big spans 37, small ones some 15 behind them, merge 12); 16 of 16384
// with up to 2000, 32 / 32 heads, 100; 3 groups of 11 with up to 5 new tokens, 20 / 4 heads of 64, 37; 8
// questions of up to 200 tokens on 16384 181, 1160 TFLOP/s of what they cannot do without.
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
// Units of a warp's run at least, where there are few.  (us in a graph with 3, 6 and 12: four forks
// of 1024 tokens 17, 19, 21; two of 32768 on 8 kv heads, which have many parts then, 51, 51, 47)
constexpr int kMinUnits = 3;
// The start of a span on a kv head counts as that many units, its rows and sums being
// what they cost: runs of equal units then take equal time.  (Of small ones 0, 2, 4: three groups
// 44, 41, 41 us; of big ones, kBigStart, 1, 3, 5: 8 questions on 16384 tokens 243, 182, 186)
constexpr int kSmallStart = 2;
// From kDynamic units a warp on, a quarter of them is cut into runs (kShort a warp) that the
// warps take as they become free: SMs differ, by their distance from the memory, in what
// they get through.  (16 forks of 16384 tokens on 32 kv heads 109 us without, 107 with; 64 forks of
// 2048 tokens, at 13 units a warp, 40 without, 51 with)
constexpr int kDynamic = 24, kShort = 2;
// Groups' prefixes are streamed whatever their rows where that is no more than so many
// units a warp: the tcgen05 kernel takes 20 us to begin with.  (8, 16 and 32: 64 forks of 2048
// tokens on 8 kv heads 46, 40, 40 us; three groups of some 170 rows and up to 9000 tokens 41, 41, 69)
constexpr int kFewUnits = 16;

struct SharedArgs {
    Attn a;
    const int *cu_groups;        // [n_groups + 1]
    const int *prefix_lens;      // [n_groups]
    int n_groups;
    int small_rows;              // groups of up to that many rows are small spans
    long long few;               // all groups are, if that is no more units than that
    int cap_big, cap_small;      // spans of groups at most
    int own_cap;                 // sequences' own spans, at most
    int warps;                   // of the streaming kernel
    int psh;                     // log2(page size)
    bool beside;                 // big spans' kernel runs before the small ones', which begin as its CTAs end
    unsigned long long token;    // the call's own number, which no memory holds by chance
    // scratch
    Span *tiles_small;           // [...]
    long long *off_small;        // [... + 1] units before each (and kSmallStart), times the kv heads
    int *rep;                    // [n_groups] the sequence whose pages are read (num_seqs: none, -1: a wrong group)
    int *at;                     // [n_groups] its first span (among those of groups) << 1 | big, or -1
    int *small_first, *small_last;  // [... * Hkv] the runs that the span on the kv head lies in
    float *small_o;              // [... * Hkv + runs][kSmallRows][D] partial sums, as part_o
    float2 *small_ml;            // [... * Hkv + runs][kSmallRows]
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
    __shared__ long long warps[4][32], s_units;
    __shared__ int s_cu[HELD ? kHeld + 1 : 1], s_len[HELD ? kHeld : 1], s_grp[HELD ? kHeld + 1 : 1];
    __shared__ int s_pre[HELD ? kHeld : 1], s_rep[HELD ? kHeld : 1], s_at[HELD ? kHeld : 1];
    const Attn &a = x.a;
    const Cache &c = a.c;
    after_previous();
    let_next();  // (not sooner: the next kernels would be brought in while a call before merges, 73 us for 69)
    const int tid = threadIdx.x, ns = c.num_seqs, ng = x.n_groups, G = a.G, Hkv = c.Hkv;
    if (HELD) {
        for (int i = tid; i <= ns; i += T) {
            s_cu[i] = c.cu[i];
            if (i < ns) s_len[i] = c.lens[i];
        }
        for (int i = tid; ng > 0 && i <= ng; i += T) {
            s_grp[i] = x.cu_groups[i];
            if (i < ng) s_pre[i] = x.prefix_lens[i];
        }
        __syncthreads();
    }
    auto cu = [&](int i) { return HELD ? s_cu[i] : c.cu[i]; };
    auto grp = [&](int i) { return HELD ? s_grp[i] : x.cu_groups[i]; };
    auto pre = [&](int i) { return HELD ? s_pre[i] : x.prefix_lens[i]; };
    int *rep = HELD ? s_rep : x.rep, *at = HELD ? s_at : x.at;
    auto sync = [&] {
        if (!HELD) __threadfence_block();
        __syncthreads();
    };
    auto seq = [&](int b, Seq &s) { return c.check(cu(b), cu(b + 1), HELD ? s_len[b] : c.lens[b], s); };
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
    // and one whose prefix ends on another page than the lender's: what the groups were
    // made of has changed since (a load a member: 1 us; taken in the loop above, no less)
    for (int b = tid; !none && b < ns; b += T) {
        Seq s;
        const int g = group_of(b);
        if (g < 0 || seq(b, s) != kSeqOk) continue;
        const int l = HELD ? *(volatile const int *)(rep + g) : __ldcg(rep + g), page = pre(g) / c.ps - 1;
        if (l < 0 || l == b || page < 0) continue;
        if (c.table[(size_t)b * c.max_pages + page] != c.table[(size_t)l * c.max_pages + page])
            atomicMin(rep + g, -1);
    }
    sync();
    // units of all groups, were they streamed
    auto lent = [&](int g, int &rows) {  // the sequence that lends its pages, and the group's rows; or -1
        const int l = HELD ? rep[g] : __ldcg(rep + g);  // (where the atomics left it)
        rows = l >= 0 && l < ns ? (cu(grp(g + 1)) - cu(grp(g))) * G : 0;
        return l >= 0 && l < ns && pre(g) > 0 ? l : -1;
    };
    if (tid == 0) s_units = 0;
    __syncthreads();
    {
        long long units = 0;
        for (int g = tid; g < ng; g += T) {
            int rows;
            if (lent(g, rows) >= 0)
                units += (long long)((rows + kSmallRows - 1) / kSmallRows) * Hkv * ((pre(g) + kUnit - 1) / kUnit);
        }
        if (units) atomicAdd(reinterpret_cast<unsigned long long *>(&s_units), (unsigned long long)units);
    }
    __syncthreads();
    const int small_rows = s_units <= x.few ? 1 << 30 : x.small_rows;
    // a group's spans: how many, and key tiles or units of each
    struct Lot {
        int lender, rows, n, tile, big;
        long long units;
    };
    auto lot_of = [&](int g) {
        Lot l = {-1, 0, 0, 1, 0, 0};
        if (g >= ng) return l;
        l.lender = lent(g, l.rows);
        if (l.lender < 0) return l;
        l.big = l.rows > small_rows;
        l.tile = l.big ? kJobRows : kSmallRows;
        l.n = (l.rows + l.tile - 1) / l.tile;
        const int p = pre(g);
        l.units = (long long)Hkv * (l.big ? (p + kBigKeys - 1) / kBigKeys + kBigStart : (p + kUnit - 1) / kUnit + kSmallStart);
        return l;
    };
    // where they begin (more than there is room for: from offsets that overlap)
    long long ng_spans[2] = {0, 0};
    for (int g0 = 0; g0 < ng; g0 += T) {
        const int g = g0 + tid;
        const Lot l = lot_of(g);
        if (g < ng && (HELD ? rep[g] : __ldcg(rep + g)) < 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        long long v[2] = {l.big ? l.n : 0, l.big ? 0 : l.n}, total[2];
        block_scan<T>(v, warps, total);
        if (g < ng) {
            const long long end = l.big ? ng_spans[0] + v[0] : ng_spans[1] + v[1];
            at[g] = l.n > 0 && end <= (l.big ? x.cap_big : x.cap_small) ? (int)(end - l.n) << 1 | l.big : -1;
        }
        ng_spans[0] += total[0];
        ng_spans[1] += total[1];
    }
    sync();
    // the sequences' own
    const int kind = a.chunk ? 0 : 1, tile_rows = a.chunk ? kJobRows : kSmallRows;
    const int unit = a.chunk ? kBigKeys : kUnit, start = a.chunk ? kBigStart : kSmallStart;
    Span *tiles = a.chunk ? a.tiles_big : x.tiles_small;
    long long *off = a.chunk ? a.off_big : x.off_small;
    long long own = 0, units = 0;
    for (int b0 = 0; b0 < ns; b0 += T) {
        const int b = b0 + tid;
        long long v[2] = {0, 0}, total[2];
        Seq s;
        Span t;
        int rows = 0;
        if (b < ns && seq(b, s) == kSeqOk) {
            const int g = group_of(b), lot = g >= 0 ? at[g] : -1;
            t.b = b;
            t.full = 0;
            t.key0 = lot >= 0 ? pre(g) : 0;
            t.pdelta = s.len - s.n - s.row0;
            t.group_row = lot >= 0 ? cu(grp(g)) * G : 0;
            t.group_span = lot;
            t.pad = t.pads[0] = t.pads[1] = 0;
            rows = s.n * G;
            v[0] = (rows + tile_rows - 1) / tile_rows;
            for (int r = 0; r < rows; r += tile_rows)
                v[1] += (s.len - s.n + (min(r + tile_rows, rows) - 1) / G - t.key0) / unit + 1 + start;
            v[1] *= Hkv;
        }
        const long long mine_n = v[0], mine_u = v[1];
        block_scan<T>(v, warps, total);
        long long i = own + v[0] - mine_n, u = units + v[1] - mine_u;
        for (int r = 0; r < rows && i < x.own_cap; r += tile_rows, ++i) {
            t.row0 = s.row0 * G + r;
            t.nrows = min(rows - r, tile_rows);
            t.key_end = (t.row0 + t.nrows - 1) / G + t.pdelta + 1;
            tiles[i] = t;
            u += (long long)Hkv * ((t.key_end - t.key0 + unit - 1) / unit + start);
            off[i + 1] = u;
        }
        own += total[0];
        units += total[1];
    }
    if (own > x.own_cap) {  // (from offsets that overlap)
        own = x.own_cap;
        sync();
        units = off[own];
    }
    // the groups' spans behind them
    long long n[2] = {kind ? 0 : own, kind ? own : 0}, un[2] = {kind ? 0 : units, kind ? units : 0};
    const long long own_of[2] = {n[0], n[1]};
    for (int g0 = 0; g0 < ng; g0 += T) {
        const int g = g0 + tid;
        const Lot l = lot_of(g);
        long long v[4] = {l.big ? l.n : 0, l.big ? 0 : l.n, l.big ? l.n * l.units : 0, l.big ? 0 : l.n * l.units}, total[4];
        block_scan<T>(v, warps, total);
        const int k = l.big ? 0 : 1;
        const long long i0 = n[k] + (l.big ? v[0] : v[1]) - l.n, u0 = un[k] + (l.big ? v[2] : v[3]) - l.n * l.units;
        const long long room = own_of[k] + (l.big ? x.cap_big : x.cap_small);
        Span *to = l.big ? a.tiles_big : x.tiles_small;
        long long *ends = l.big ? a.off_big : x.off_small;
        for (int i = 0; i < l.n && i0 + i < room; ++i) {
            Span t;
            t.row0 = cu(grp(g)) * G + i * l.tile;
            t.nrows = min(l.rows - i * l.tile, l.tile);
            t.b = l.lender;
            t.full = 1;
            t.key0 = 0;
            t.key_end = pre(g);
            t.pdelta = t.group_row = 0;
            t.group_span = -1;
            t.pad = t.pads[0] = t.pads[1] = 0;
            to[i0 + i] = t;
            ends[i0 + i + 1] = u0 + l.units * (i + 1);
        }
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            n[z] += total[z];
            un[z] += total[2 + z];
        }
    }
    if (tid == 0) a.off_big[0] = x.off_small[0] = 0;
    const long long room[2] = {own_of[0] + x.cap_big, own_of[1] + x.cap_small};
    if (n[0] > room[0] || n[1] > room[1]) {
        sync();
        if (n[0] > room[0]) n[0] = room[0], un[0] = a.off_big[room[0]];
        if (n[1] > room[1]) n[1] = room[1], un[1] = x.off_small[room[1]];
    }
    if (tid == 0) {
        SpanHead h;
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            h.units[z] = un[z];
            h.spans[z] = (int)n[z];
            h.own[z] = (int)own_of[z];
        }
        h.taken = h.pad[0] = h.pad[1] = h.pad[2] = 0;
        h.ready = h.pads = 0;
        *a.head = h;
    }
    if (x.beside) {  // (every thread's part of it, and all that was before it on the stream)
        __syncthreads();
        if (tid == 0) ptx::st_release(&a.head->ready, x.token);
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
    __shared__ int s_abort, s_ready;
    const Attn &a = x.a;
    const Cache &c = a.c;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n8 = lane >> 2, c4 = lane & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStreamWarps; ++i)
            for (int s = 0; s < ST; ++s) ptx::mbar_init(ptx::saddr(&s_bar[i][s]), 1);
        s_abort = 0;
        s_ready = x.beside && ptx::ld_acquire(&a.head->ready) == x.token;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    // Behind the plan.  Where the big spans' kernel lies between them, this one needs nothing of
    // its results, so that it only has to end behind it (the merge waits for this one's end).
    // It is let in once all CTAs of that one have waited for the plan; but that orders no
    // memory, so the plan is taken as made where its token says so (in a row of release, acquire
    // and barrier that what was before the plan is in too), and else by waiting for all.
    const bool early = s_ready;
    if (early) asm volatile("fence.proxy.async.global;" ::: "memory");  // (for the bulk copies too)
    else after_previous();
    let_next();
    ptx::Ctl ctl{&s_abort, a.status, kDefaultWaitLimit};
    const uint32_t raw = ptx::saddr(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t ring = base + warp * ST * R::kStage, bars = ptx::saddr(&s_bar[warp][0]);
    const uint8_t *mine = smem_raw + (ring - raw);
    const int gw = blockIdx.x * kStreamWarps + warp, G = a.G, Hkv = c.Hkv, ps = c.ps;
    const int spans = a.head->spans[1];
    const long long total = a.head->units[1], most = (total + kMinUnits - 1) / kMinUnits;
    // the short runs are the first ones, of sequences' own keys: of few parts' rows
    const bool dynamic = total > (long long)x.warps * kDynamic;
    const int shorts = dynamic ? x.warps * kShort : 0;
    const long long cut = dynamic ? total / 4 : 0;  // the units of the short runs
    const int runs = shorts + (int)(most < x.warps ? most : x.warps);
    auto begin = [&](int r) {
        return r < shorts ? cut * r / shorts : cut + (total - cut) * (r - shorts) / (runs - shorts);
    };
    int issued = 0, used = 0;  // stages so far
    for (int run = shorts + gw, next = 0; run < runs; run = next) {
        if (dynamic && lane == 0) next = atomicAdd(&a.head->taken, 1);
        const long long u0 = begin(run);
        const int n = (int)(begin(run + 1) - u0);
        int w = span_of_unit(x.off_small, spans, u0, lane);
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
                    const int page = c.table[(size_t)s.b * c.max_pages + (key >> x.psh)];
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
                    qr[i][h] = live ? *reinterpret_cast<const uint4 *>(src + 64 * (i >> 1) + 8 * (i & 1))
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
            break;
        }
        next = __shfl_sync(0xffffffffu, next, 0);
        if (next >= shorts) break;
    }
    if (early) after_previous();
}

// ----------------------------------------------------------------------------
// merge
// ----------------------------------------------------------------------------
// A CTA takes up to `most` rows of a sequence's own span on a kv head, whose parts and whose
// group's it looks up once.  Its threads are teams of TEAM, a row each; W of them to a row,
// every W-th part each, where rows are few (they have many parts then).  Teams of 16 for chunks,
// of 32 for small spans: there the same rows have more warps, with half the columns a lane.
constexpr int kMergeThreads = 256, kMergeRows = 32;

template <int D, int TEAM>
__global__ void __launch_bounds__(kMergeThreads, TEAM == 16 ? 3 : 4) merge_spans_kernel(SharedArgs x, int most) {
    constexpr int V = D / TEAM, U = 4, kTeams = kMergeThreads / TEAM;
    __shared__ __align__(16) float s_acc[kTeams][D];
    __shared__ float s_m[kTeams], s_l[kTeams];
    const Attn &a = x.a;
    after_previous();
    let_next();
    if (x.beside && threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) a.head->ready = 0;  // (a replay has the same token)
    const int team = threadIdx.x / TEAM, lane = threadIdx.x % TEAM, G = a.G, Hkv = a.c.Hkv;
    const bool chunk = a.chunk;
    // (a span behind the last one is some memory of the scratch)
    const int w = (int)blockIdx.x / Hkv, hk = blockIdx.x % Hkv;
    const Span s = (chunk ? a.tiles_big : x.tiles_small)[w];
    const int groups = a.head->own[chunk ? 0 : 1], big_groups = chunk ? groups : a.head->own[0], small_groups = a.head->own[1];
    if (w >= groups) return;
    const int r0 = blockIdx.y * most, rows = min(s.nrows - r0, most);
    if (rows <= 0) return;
    const int slots = rows > 4 ? 8 : rows > 2 ? 4 : rows > 1 ? 2 : 1;  // rows at a time
    const int W = rows > 8 || kTeams == slots ? 1 : kTeams / slots;    // teams to a row
    const int part = team % W;
    for (int ri = team / W; ri < (W > 1 ? kTeams / W : rows); ri += kTeams / W) {
        const bool live = ri < rows;
        const int row = s.row0 + r0 + ri;
        float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
        for (int k = 0; k < V; ++k) acc[k] = 0.f;
        bool bad = false;
        // its parts: of its group's span, then of its own one, those of a run (or CTA) each
        int np = 0, n = 0;
        const float *o[2] = {nullptr, nullptr};
        const float2 *ml[2] = {nullptr, nullptr};
        size_t first[2] = {0, 0};
        int rows_of[2] = {0, 0};
        auto parts = [&](int which, bool big, int e, int r) {
            const int c0 = max((big ? a.c_first : x.small_first)[e], 0);
            const int c1 = min((big ? a.c_last : x.small_last)[e], (big ? a.ctas : x.warps * (1 + kShort)) - 1);
            o[which] = big ? a.part_o : x.small_o;
            ml[which] = big ? a.part_ml : x.small_ml;
            rows_of[which] = big ? kJobRows : kSmallRows;
            first[which] = ((size_t)e + c0) * rows_of[which] + r;
            return max(c1 - c0 + 1, 0);
        };
        if (live) {
            if (s.group_span >= 0) {
                const bool big = s.group_span & 1;
                const int at = row - s.group_row, tile = big ? kJobRows : kSmallRows;
                np = parts(0, big, ((big ? big_groups : small_groups) + (s.group_span >> 1) + at / tile) * Hkv + hk, at % tile);
            }
            n = np + parts(1, chunk, w * Hkv + hk, r0 + ri);
        }
        for (int i = part; i < n; i += W * U) {
            float2 z[U];
            float v[U][V];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                z[j] = make_float2(-INFINITY, 0.f);
                const int k = i + W * j;
                const bool of_group = k < np;
                if (k < n) {
                    const size_t p = of_group ? first[0] + (size_t)k * rows_of[0] : first[1] + (size_t)(k - np) * rows_of[1];
                    z[j] = (of_group ? ml[0] : ml[1])[p];
                    const float *src = (of_group ? o[0] : o[1]) + p * D + lane * V;
#pragma unroll
                    for (int d = 0; d < V; d += 2)
                        *reinterpret_cast<float2 *>(&v[j][d]) = *reinterpret_cast<const float2 *>(src + d);
                }
            }
            float top = M;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                bad |= z[j].y < 0.f;
                if (z[j].y == 0.f) z[j].x = -INFINITY;  // no part, or one without a key for this row
                top = fmaxf(top, z[j].x);
            }
            const float ref = top == -INFINITY ? 0.f : top, f = mma::fast_exp2(M - ref);
            M = top;
            L *= f;
#pragma unroll
            for (int d = 0; d < V; ++d) acc[d] *= f;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (z[j].y == 0.f) continue;  // (a sum that is not a number stays in)
                const float g = mma::fast_exp2(z[j].x - ref);
                L = fmaf(z[j].y, g, L);
#pragma unroll
                for (int d = 0; d < V; ++d) acc[d] = fmaf(v[j][d], g, acc[d]);
            }
        }
        if (W > 1) {  // (one round: every team is here)
#pragma unroll
            for (int k = 0; k < V; ++k) s_acc[team][lane * V + k] = acc[k];
            if (lane == 0) {
                s_m[team] = M;
                s_l[team] = bad ? -1.f : L;
            }
            __syncthreads();
            if (!live || part) return;
            M = -INFINITY;
            L = 0.f;
            bad = false;
            for (int i = team; i < team + W; ++i) {
                M = fmaxf(M, s_m[i]);
                bad |= s_l[i] < 0.f;
            }
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
            for (int i = team; i < team + W; ++i) {
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
    const size_t ng = x->n_groups, nb = (size_t)x->cap_big + (a.chunk ? x->own_cap : 0);
    const size_t nm = (size_t)x->cap_small + (a.chunk ? 0 : x->own_cap);
    a.head = static_cast<SpanHead *>(take(sizeof(SpanHead)));
    a.tiles_big = static_cast<Span *>(take(sizeof(Span) * nb));
    a.off_big = static_cast<long long *>(take(8 * (nb + 1)));
    x->tiles_small = static_cast<Span *>(take(sizeof(Span) * nm));
    x->off_small = static_cast<long long *>(take(8 * (nm + 1)));
    x->rep = static_cast<int *>(take(4 * ng));
    x->at = static_cast<int *>(take(4 * ng));
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
    const long long lent = groups ? rows / kSmallRows + groups : 0;  // small spans of groups, at most
    x->few = a.chunk ? -1 : (long long)x->warps * kFewUnits;
    // no group is big where even a prefix as long as the table is few units
    const bool never = !a.chunk && lent * a.c.Hkv * ((long long)a.c.max_pages * a.c.ps / kUnit) <= x->few;
    // (with up to as many groups as have more rows than a small span, where those are streamed)
    const long long large = a.chunk ? groups : groups < rows / (kSmallRows + 1) ? groups : rows / (kSmallRows + 1);
    const long long big = large && !never ? rows / kJobRows + large : 0;
    const long long small = a.chunk ? 0 : lent;
    if ((big + own) * a.c.Hkv >= (1ll << 30) || (small + own) * a.c.Hkv >= (1ll << 30)) return MOBA_ERR_UNSUPPORTED;
    x->cap_big = (int)big;
    x->cap_small = (int)small;
    x->own_cap = (int)own;
    return MOBA_OK;
}

cudaError_t launch_plan(const SharedArgs &x, cudaStream_t st) {
    note_launches(1);
    const int most = x.a.c.num_seqs > x.n_groups ? x.a.c.num_seqs : x.n_groups;
    return most <= 128     ? launch_after(plan_spans_kernel<128, true>, dim3(1), dim3(128), 0, st, x)
           : most <= kHeld ? launch_after(plan_spans_kernel<1024, true>, dim3(1), dim3(1024), 0, st, x)
                           : launch_after(plan_spans_kernel<1024, false>, dim3(1), dim3(1024), 0, st, x);
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
    const Attn &a = x.a;
    const long long spans = (long long)x.own_cap * a.c.Hkv, fill = 4 * (long long)a.ctas;
    const int rows = a.chunk ? kJobRows : a.c.max_new * a.G < kSmallRows ? a.c.max_new * a.G : kSmallRows;
    int most = a.chunk ? kMergeRows : rows;  // rows of a CTA: fewer where that leaves SMs without one
    while (!a.chunk && most > 1 && spans * ((rows + most - 1) / most) < fill) most = (most + 1) / 2;
    const dim3 grid((unsigned)spans, (rows + most - 1) / most);
    note_launches(1);
    return a.chunk ? launch_after(merge_spans_kernel<D, 16>, grid, dim3(kMergeThreads), 0, st, x, most)
                   : launch_after(merge_spans_kernel<D, 32>, grid, dim3(kMergeThreads), 0, st, x, most);
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
    x.beside = x.cap_big && !a.chunk;
    x.token = call_token();
    cudaError_t e = launch_plan(x, st);
    if (e == cudaSuccess && (x.cap_big || a.chunk)) e = launch_chunk_spans(a, st);
    if (e == cudaSuccess && !a.chunk) e = D == 64 ? launch_small<64>(x, st) : launch_small<128>(x, st);
    if (e == cudaSuccess) e = D == 64 ? launch_merge<64>(x, st) : launch_merge<128>(x, st);
    if (own) {
        const cudaError_t f = cudaFreeAsync(own, st);
        if (e == cudaSuccess) e = f;
    }
    return cuda_result(e);
}
