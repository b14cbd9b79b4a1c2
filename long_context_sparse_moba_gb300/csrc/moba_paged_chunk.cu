// moba_paged_chunk.cu -- attention of chunks of many query rows over a paged
// cache on the sm_103a tensor cores (tcgen05.mma, accumulators in tensor memory,
// K/V pages staged by TMA).
//
// Pages: "When a MoBA reproduction will not run" (mhpq.cn/news/582794) section
// 3.3 (the selected blocks of all queries batched before the attention) and
// "MOBA mixture of block attention for server-side long context"
// (hncyxsy.com/news/197418) section 3 (own block forced, causal inside it).
//
// A row is a (new token, query head of a kv head's group); the rows of one kv
// head are numbered token * G + head, so that a job's 256 rows share its keys
// whatever the group size.  Jobs:
//   with selection: (1) up to 256 rows that selected one past block of one kv
//     head, from its list; the last rows of a list, where they are 128 at most,
//     share a job with another list's, each with its own keys, so that one Q
//     tile's MMAs still run under the other's softmax; (2) up to 256 consecutive
//     rows with the keys of their own blocks.  Each writes, for a row and slot, a normalised partial
//     output and its log2-sum-exp; the merge kernel joins a row's slots.
//     Partials are fp16 with a power-of-two scale per row and 64 columns: half
//     the bytes of fp32, and 2^-11 of a value is a fraction of the rounding of
//     the result (bf16 partials would double its error);
//   all blocks: 256 consecutive rows with every key up to them.  The key tiles
//     of all jobs form one sequence that is cut into equal runs, one per CTA; a
//     job that falls into several runs leaves fp32 partial sums.
//
// With selection, the CTAs start as the gate's leave and work off equal shares of
// (2), which need no list, while the plan and scatter kernels make the lists (15 us of
// a call of 200 at 4096 tokens x 32 heads of 128 over 32768 keys).  A mark in the ring of
// job descriptors then has every role wait for those kernels.
//
// Persistent, one CTA per SM, 12 warps:
//   warp 0   K pages by TMA (one lane), warp 10 V pages, into rings of tiles;
//   warp 1   allocates TMEM; an elected lane issues, for the two 128-row tiles g of a
//            job, PV_0(j-1), S_0(j), PV_1(j-1), S_1(j): one tile's MMAs run
//            while the other tile's softmax works;
//   warps 2..9  softmax: thread r owns row r of its tile.  The offset mu is
//            raised, to a whole number, only when the maximum exceeds it by more
//            than 8, so that a rescale is by an exact power of two and rare.
//            They gather the next job's query rows as soon as the MMAs have
//            released Q, and write the results;
//   warp 11  one lane hands job descriptors to the others, three ahead.
// Keys that no row of a job sees (behind its last row, possibly never written)
// are zeroed in the V tile before its product; in K their scores are masked.
// Bound: tensor and softmax in turn where jobs are long: 2048 rows x 32 heads over
// 32768 keys of 128 take 719 us in this kernel alone, 800 us in a row of
// calls, 1340 TFLOP/s, 0.70 of the burst peak.  168 registers a thread is all that 384
// threads leave: over all blocks the softmax spills 40 to 52 bytes, with lists nothing.
// Job boundaries where they are short: 4096 tokens x 32 heads, three blocks of 512
// (four tiles a job) 100 us behind the lists; blocks of 128 are one tile a job.
// Every mbarrier wait is bounded: one that runs out sets MOBA_ERR_TIMEOUT in the
// status word and an abort flag that makes every role leave; copies and MMAs
// in flight are awaited before the CTA frees its tensor memory.
#include <atomic>

#include "moba_paged_attn.cuh"
#include "moba_ptx.cuh"

namespace moba {
namespace paged {
namespace {

using namespace ptx;

constexpr int kM = 128;          // rows per Q tile
constexpr int kG = 2;            // Q tiles per job
constexpr int kThreads = 384;
constexpr int kTmemCols = 512;
constexpr int kJobs = 3;         // descriptors in flight
constexpr int kBadSlots = 8;

__device__ __forceinline__ bool elected() {
    uint32_t e;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(e));
    return e != 0;
}
// A commit and an arrival by one elected lane of a warp that runs them as one.
__device__ __forceinline__ void one_commit(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
        : "memory");
}
__device__ __forceinline__ void one_arrive(uint32_t bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(bar)
        : "memory");
}

// One Q tile's share of a job.
struct Half {
    int b, hk;
    int rbase;       // own: first row; list: first entry
    int nrows;       // of its 128
    int key0;        // position of the keys' first tile
    int te;          // tiles that it visits
    int rlo, rn;     // list: the sequence's rows [rlo, rlo + rn)
};
enum { kNoJob = 0, kAJob = 1, kLists = 2 };
enum { kCausal = 1, kFull = 2 };
struct Job {
    Half h[kG];
    int valid;       // kNoJob: leave; kLists: no job, the kernels before have to end first
    int own;         // consecutive rows (else lists): kCausal, or kFull (keys whole)
    int pair;        // the Q tiles have rows of two lists, and their own keys each
    int key_end;     // own: keys from here on are seen by no row
    int lo, nt;      // first key tile of this job's part, and how many
    int pdelta;      // own: position of a row = its token + pdelta
    int whole;       // all blocks: the part is the whole job
    int slot;        // all blocks: partial slot
    int pad[3];
};

struct ChunkArgs {
    Attn a;
    int psh;         // log2(page size)
    long long wait_limit;
};

template <int D, int N>
struct Smem {
    static constexpr int NB = D / 64;                    // 64-dim boxes per row
    static constexpr int kStages = N == 128 ? 2 : 4;
    static constexpr uint32_t kQBox = kM * 128;
    static constexpr uint32_t kKVBox = N * 128;
    static constexpr uint32_t kTileBytes = NB * kKVBox;
    static constexpr uint32_t kQ = 0;
    static constexpr uint32_t kK = kQ + kG * NB * kQBox;
    static constexpr uint32_t kV = kK + kStages * kTileBytes;
    static constexpr uint32_t kStage = kV + kStages * kTileBytes;  // 4 KB per softmax warp
    static constexpr uint32_t kEnd = kStage + 4 * kG * 4096;
    static constexpr int kBarQ = 0, kBarQE = kBarQ + kG, kBarKF = kBarQE + kG,
                         kBarKE = kBarKF + kStages, kBarVF = kBarKE + kStages,
                         kBarVE = kBarVF + kStages, kBarS = kBarVE + kStages, kBarP = kBarS + kG,
                         kBarPV = kBarP + kG, kBarDrain = kBarPV + kG,
                         kBarJF = kBarDrain + 1, kBarJE = kBarJF + kJobs, kNumBars = kBarJE + kJobs;
    static constexpr uint32_t kSlot = kNumBars * 8;      // TMEM address, abort flag
    static constexpr uint32_t kBad = kSlot + 8;
    static constexpr uint32_t kJob = (kBad + 4 * kBadSlots + 15) & ~15u;
    static constexpr uint32_t kMisc = kJob + kJobs * sizeof(Job);
    static constexpr uint32_t kNeed = kEnd + 1008 + kMisc;
    static_assert(kNeed <= 227 * 1024, "shared memory per CTA");
    static constexpr uint32_t kRequest = kNeed > 120 * 1024 ? kNeed : 120 * 1024;
};

// The job of the 256-row tile x of sequence b on kv head hk, all its key tiles.
template <int N>
__device__ __forceinline__ void own_job(const Attn &a, const Seq &s, int b, int hk, int x, Job &J) {
    const int r0 = x * kJobRows, nrows = min(kJobRows, s.n * a.G - r0);
    J.valid = kAJob;
    J.own = kCausal;
    J.pair = 0;
    J.pdelta = s.len - s.n - s.row0;
    const int pf = s.len - s.n + r0 / a.G, pl = s.len - s.n + (r0 + nrows - 1) / a.G;
    const int key0 = a.dense ? 0 : pf / a.c.bs * a.c.bs;
    J.key_end = pl + 1;
    J.lo = 0;
    J.nt = (pl - key0) / N + 1;
    J.whole = 1;
    J.slot = 0;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        J.h[g].b = b;
        J.h[g].hk = hk;
        J.h[g].rbase = s.row0 * a.G + r0 + g * kM;
        J.h[g].nrows = min(max(nrows - g * kM, 0), kM);
        J.h[g].key0 = key0;
        J.h[g].rlo = J.h[g].rn = 0;
    }
}

// A span as a job, all its key tiles.
template <int N>
__device__ __forceinline__ void span_job(const Span &s, Job &J) {
    J.valid = kAJob;
    J.own = s.full ? kFull : kCausal;
    J.pair = 0;
    J.pdelta = s.pdelta;
    J.key_end = s.key_end;
    J.lo = 0;
    J.nt = (s.key_end - s.key0 + N - 1) / N;
    J.whole = 0;
    J.slot = 0;
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        J.h[g].b = s.b;
        J.h[g].hk = 0;
        J.h[g].rbase = s.row0 + g * kM;
        J.h[g].nrows = min(max(s.nrows - g * kM, 0), kM);
        J.h[g].key0 = s.key0;
        J.h[g].rlo = J.h[g].rn = 0;
    }
}

// A Q tile's share of the part's tiles: those up to its last row.
template <int N>
__device__ __forceinline__ void own_ends(const Attn &a, Job &J) {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
        const int last = J.own == kFull ? J.key_end - 1 : (J.h[g].rbase + J.h[g].nrows - 1) / a.G + J.pdelta;
        J.h[g].te = J.h[g].nrows > 0 ? min(max((last - J.h[g].key0) / N + 1 - J.lo, 0), J.nt) : 0;
    }
}

// Up to 128 rows of a list, from entry `start` on, as a Q tile's share.
template <int N>
__device__ __forceinline__ void list_half(const Attn &a, int l, int start, Half &h) {
    const int lb = a.list_off[l];
    h.hk = l % a.c.Hkv;
    const int bc = l / a.c.Hkv;
    h.b = bc / a.n_max;
    h.rbase = lb + start;
    h.nrows = min(max(min(a.counts[l], (int)a.list_cap - lb) - start, 0), kM);
    h.key0 = (bc - h.b * a.n_max) * a.c.bs;
    h.te = h.nrows > 0 ? a.c.bs / N : 0;
    Seq s;
    a.c.seq(h.b, s);
    h.rlo = s.row0 * a.G;
    h.rn = s.n * a.G;
}

// SPANS (with DENSE): jobs from spans; every part of one leaves partial sums.
template <int D, int N, bool DENSE, bool SPANS>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmap_k,
                 const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ ChunkArgs ca) {
    using L = Smem<D, N>;
    constexpr int ST = L::kStages;
    const Attn &a = ca.a;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = saddr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t misc = base - raw >= L::kMisc ? raw : base + L::kEnd;
    uint8_t *gmisc = smem_raw + (misc - raw);
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be uniform)
    const uint32_t sQ = base + L::kQ, sK = base + L::kK, sV = base + L::kV;
    auto bar = [&](int i) -> uint32_t { return misc + 8u * (uint32_t)i; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gmisc + L::kSlot);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(gmisc + L::kSlot + 4);
    volatile int *bad_job = reinterpret_cast<volatile int *>(gmisc + L::kBad);
    Job *ring = reinterpret_cast<Job *>(gmisc + L::kJob);
    Ctl ctl{abort_flag, a.status, ca.wait_limit};

    if (tid == 0) {
        for (int g = 0; g < kG; ++g) {
            mbar_init(bar(L::kBarQ + g), kM);  // an asynchronous arrival per gathering thread
            mbar_init(bar(L::kBarQE + g), 1);
            mbar_init(bar(L::kBarS + g), 1);
            mbar_init(bar(L::kBarP + g), 4);
            mbar_init(bar(L::kBarPV + g), 1);
        }
        for (int s = 0; s < ST; ++s) {
            mbar_init(bar(L::kBarKF + s), 1);
            mbar_init(bar(L::kBarKE + s), 1);
            mbar_init(bar(L::kBarVF + s), 1);
            mbar_init(bar(L::kBarVE + s), 1);
        }
        for (int s = 0; s < kJobs; ++s) {
            mbar_init(bar(L::kBarJF + s), 1);
            mbar_init(bar(L::kBarJE + s), 4 * kG + 3);  // softmax warps, producers, MMA lane
        }
        mbar_init(bar(L::kBarDrain), 1);
        for (int i = 0; i < kBadSlots; ++i) bad_job[i] = 0;
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    if (tid == 0)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
    if (tid == 320)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
    if (DENSE) after_previous();
    let_next();  // (SPANS: the small spans' kernel, which goes by the plan's token, not by this)

    if (warp == 11) {
        // ================= job descriptors =================
        // (spans: the run's first one is looked for by the whole warp)
        int first_span = 0;
        if constexpr (SPANS) {
            const long long total = a.head->units[0], runs = total < (long long)gridDim.x ? total : (long long)gridDim.x;
            if ((long long)blockIdx.x < runs)
                first_span = span_of_unit(a.off_big, a.head->spans[0], total * blockIdx.x / runs, lane);
        }
        if (lane == 0) {
            int n = 0;
            auto hand = [&](const Job &J) -> bool {
                const int s = n % kJobs;
                if (n >= kJobs && !wait_bar(bar(L::kBarJE + s), (n / kJobs - 1) & 1, ctl)) return false;
                ring[s] = J;
                mbar_arrive(bar(L::kBarJF + s));
                ++n;
                return true;
            };
            bool go = true;
            Job J;
            Seq sq;
            if (DENSE) {
                const int tiles = SPANS ? a.head->spans[0] : a.own_off[a.c.num_seqs];
                const long long *off = SPANS ? a.off_big : a.unit_off;
                int open = -1;
                const long long total = SPANS ? a.head->units[0] : off[tiles];
                const long long runs = total < (long long)gridDim.x ? total : (long long)gridDim.x;
                if ((long long)blockIdx.x < runs) {
                    long long u = total * blockIdx.x / runs;
                    const long long u1 = total * (blockIdx.x + 1) / runs;
                    int w = first_span, hi = SPANS ? w : tiles - 1;  // largest row tile that starts at or before u
                    while (w < hi) {
                        const int mid = (w + hi + 1) >> 1;
                        if (off[mid] <= u) w = mid; else hi = mid - 1;
                    }
                    while (go && u < u1) {
                        if constexpr (SPANS) {
                            const Span s = a.tiles_big[w];
                            span_job<N>(s, J);
                        } else {
                            const int b = seq_of_tile(a, w);
                            a.c.seq(b, sq);
                            own_job<N>(a, sq, b, 0, w - a.own_off[b], J);
                        }
                        const int T = J.nt;
                        for (; go && u < u1 && u < off[w + 1];) {
                            const long long in = u - off[w];
                            if constexpr (SPANS) {
                                // (the first units of a span on a kv head stand for its start)
                                const int V = T + kBigStart, hk = (int)(in / V), v0 = (int)(in - (long long)hk * V);
                                const int take = (int)min((long long)(V - v0), u1 - u), e = w * a.c.Hkv + hk;
                                J.h[0].hk = J.h[1].hk = hk;
                                J.lo = max(v0 - kBigStart, 0);
                                J.nt = v0 + take - kBigStart - J.lo;
                                J.slot = e + blockIdx.x;
                                u += take;
                                if (J.nt <= 0) continue;
                                if (J.lo == 0) a.c_first[e] = blockIdx.x;
                                if (J.lo + J.nt == T) a.c_last[e] = blockIdx.x;
                                own_ends<N>(a, J);
                                go = hand(J);
                            } else {
                                const int hk = (int)(in / T);
                                J.h[0].hk = J.h[1].hk = hk;
                                J.lo = (int)(in - (long long)hk * T);
                                J.nt = (int)min((long long)(T - J.lo), u1 - u);
                                J.whole = J.nt == T;
                                J.slot = blockIdx.x * 2 + (J.lo == 0 ? 1 : 0);
                                own_ends<N>(a, J);
                                const int e = w * a.c.Hkv + hk;
                                if (J.lo + J.nt == T) a.c_last[e] = blockIdx.x;
                                else if (J.lo == 0) open = e;
                                go = hand(J);
                                u += J.nt;
                            }
                        }
                        ++w;
                    }
                }
                if (!SPANS) a.c_open[blockIdx.x] = open;
            } else {
                // own blocks need none of the lists: equal shares of them are worked off
                // while the kernels before make those
                const long long owns = a.c.tile_slots(a.G, kJobRows, 1) * a.c.Hkv;
                const long long shared = owns - owns % gridDim.x;
                auto own = [&](long long u) -> bool {
                    int x;
                    const int b = a.c.tile_of((int)(u / a.c.Hkv), a.G, kJobRows, 1, x);
                    if (a.c.seq(b, sq) != kSeqOk || x < 0 || (long long)x * kJobRows >= (long long)sq.n * a.G)
                        return true;
                    own_job<N>(a, sq, b, (int)(u % a.c.Hkv), x, J);
                    own_ends<N>(a, J);
                    return hand(J);
                };
                for (long long u = blockIdx.x; go && u < shared; u += gridDim.x) go = own(u);
                // every role waits for those kernels itself, however long they take: a
                // bounded wait for the next job would run while they work
                J.valid = kLists;
                if (go) go = hand(J);
                after_previous();
                // jobs: 256 rows of a list; pairs of lists' last rows, up to 128
                // each; the own blocks that are left
                const int full = a.km1 > 0 ? a.n_jobs[0] : 0, halves = a.km1 > 0 ? a.n_jobs[1] : 0;
                const int listed = full + (halves + 1) / 2;
                const long long all = listed + owns - shared;
                // jobs differ in length: taken as CTAs become free (the next one's
                // number is fetched while this one is looked up)
                long long q = atomicAdd(a.n_jobs + 2, 1);
                while (go && q < all) {
                    const long long after = atomicAdd(a.n_jobs + 2, 1);
                    if (q < listed) {
                        J.valid = kAJob;
                        J.own = 0;
                        J.key_end = 0x7fffffff;
                        J.lo = 0;
                        J.nt = a.c.bs / N;
                        J.pdelta = 0;
                        J.whole = 1;
                        J.slot = 0;
                        if (q < full) {
                            const int2 d = a.jobs[q];
                            list_half<N>(a, d.x, d.y, J.h[0]);
                            list_half<N>(a, d.x, d.y + kM, J.h[1]);
                            J.pair = 0;
                        } else {
                            const int h = 2 * (int)(q - full);
                            const int2 d = a.halves[h];
                            list_half<N>(a, d.x, d.y, J.h[0]);
                            J.pair = h + 1 < halves;
                            if (J.pair) {
                                const int2 f = a.halves[h + 1];
                                list_half<N>(a, f.x, f.y, J.h[1]);
                                // (an empty one: only where refused sequences spoilt the counts)
                                if (J.h[0].te == 0) J.h[0] = J.h[1], J.pair = 0;
                                else if (J.h[1].te == 0) J.pair = 0;
                            }
                            if (!J.pair) {
                                J.h[1] = J.h[0];
                                J.h[1].nrows = J.h[1].te = 0;
                            }
                        }
                    } else {
                        go = own(shared + q - listed);
                    }
                    if (q < listed) go = hand(J);
                    q = after;
                }
            }
            J.valid = kNoJob;
            if (go) hand(J);
        }
        __syncwarp();
    } else if (warp == 0 || warp == 10) {
        // ================= K pages (warp 0), V pages (warp 10) =================
        if (lane == 0) {
            const bool is_k = warp == 0;
            const int bfull = is_k ? L::kBarKF : L::kBarVF, bempty = is_k ? L::kBarKE : L::kBarVE;
            const uint32_t tiles = is_k ? sK : sV;
            const CUtensorMap *map = is_k ? &tmap_k : &tmap_v;
            const int ps = a.c.ps, box = min(ps, N);
            int pend[ST];
            for (int s = 0; s < ST; ++s) pend[s] = -1;
            int t = 0, n = -1;  // tiles so far, the job's number
            for (int r = 0;; ++r) {
                const int js = r % kJobs;
                if (!wait_bar(bar(L::kBarJF + js), (r / kJobs) & 1, ctl)) break;
                const Job J = ring[js];
                mbar_arrive(bar(L::kBarJE + js));
                if (J.valid == kNoJob) break;
                if (J.valid == kLists) {
                    after_previous();
                    continue;
                }
                ++n;
                bool ok = true;
                const int tiles_of_job = J.pair ? 2 * J.nt : J.nt;
                for (int j = 0; j < tiles_of_job; ++j, ++t) {
                    const int s = t % ST;
                    // (a pair's Q tiles take their tiles in turn)
                    const int g = J.pair ? j & 1 : 0, i0 = J.pair ? j >> 1 : j;
                    const int hb = g ? J.h[1].b : J.h[0].b, hk = g ? J.h[1].hk : J.h[0].hk;
                    const int p0 = (g ? J.h[1].key0 : J.h[0].key0) + (J.lo + i0) * N;
                    const int *table = a.c.table + (size_t)hb * a.c.max_pages;
                    const int nv = min(N, J.key_end - p0);  // keys that some row sees
                    const int boxes = (nv + box - 1) / box;
                    int page[N / 16];
#pragma unroll
                    for (int i = 0; i < N / 16; ++i)
                        if (i < boxes) page[i] = __ldg(table + ((p0 + i * box) >> ca.psh));
                    if (t >= ST && !wait_bar(bar(bempty + s), (t / ST - 1) & 1, ctl)) {
                        ok = false;
                        break;
                    }
                    pend[s] = -1;
                    mbar_expect_tx(bar(bfull + s), (uint32_t)(boxes * box) * 128u * L::NB);
#pragma unroll
                    for (int i = 0; i < N / 16; ++i) {
                        if (i >= boxes) continue;
                        if ((unsigned)page[i] >= (unsigned)a.c.num_pages) {
                            page[i] = 0;  // some memory of the pool; the job's results are dropped
                            if (is_k) {
                                bad_job[n % kBadSlots] = n + 1;
                                __threadfence_block();
                            }
                        }
                        const int row = (page[i] * a.c.Hkv + hk) * ps + ((p0 + i * box) & (ps - 1));
#pragma unroll
                        for (int x = 0; x < L::NB; ++x)
                            asm volatile(
                                "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::"
                                "bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
                                    tiles + s * L::kTileBytes + x * L::kKVBox + (uint32_t)(i * box) * 128u),
                                "l"(reinterpret_cast<uint64_t>(map)), "r"(bar(bfull + s)), "r"(x * 64),
                                "r"(row)
                                : "memory");
                    }
                    pend[s] = t;
                }
                if (!ok) break;
            }
            if (*abort_flag)
                for (int s = 0; s < ST; ++s)
                    if (pend[s] >= 0) drain_bar(bar(bfull + s), (pend[s] / ST) & 1, ca.wait_limit);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ================= MMA issuer =================
        // The whole warp runs the loops, with the job and the waits' results broadcast so
        // that the flow is uniform, and an elected lane issues a product's MMAs.  (One
        // lane that ran all of it took 92 cycles an MMA, 65 being the tensor core's: 895
        // us instead of 800 over all blocks.)
        auto poll = [&](int b, int parity) -> bool {
            return __all_sync(0xffffffffu, wait_poll(bar(b), parity, ctl));
        };
        auto all = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
        constexpr uint32_t idesc_s = idesc_bf16(kM, N, 0);
        constexpr uint32_t idesc_o = idesc_bf16(kM, D, 1);
        int t = 0;
        int gt[kG] = {0, 0};  // S tiles of each Q tile so far
        bool ok = true;
        // descriptors of the first tiles; the address field counts 16 bytes
        const uint64_t qd0 = sdesc(sQ, 16, 1024), kd0 = sdesc(sK, 16, 1024),
                       vd0 = sdesc(sV, L::kKVBox, 1024);
        // O_g += P_g V of tile i of Q tile g, V described by vd; P_g is in the first
        // columns of S_g (a job's first P is made after the last job's O was read)
        auto pv = [&](int g, int i, int te, uint64_t vd) -> bool {
            if (!poll(L::kBarP + g, (gt[g] + i) & 1)) return false;
            tc_fence_after();
            const uint32_t tS = tmem + g * 256, tO = tS + 128;
            const uint32_t more = i > 0;
            if (elected()) {
                tc_mma_ta(tO, tS, vd, idesc_o, more);
#pragma unroll
                for (int k = 1; k < N / 16; ++k) tc_mma_ta(tO, tS + k * 8, vd + k * 128, idesc_o, 1u);
                if (i == te - 1) tc_commit(bar(L::kBarPV + g));
            }
            __syncwarp();
            return true;
        };
        // S_g = Q_g K^T of tile i of Q tile g, K described by kd
        auto qk = [&](int g, int i, int te, uint64_t kd, int n) -> bool {
            if (i == 0) {
                if (!poll(L::kBarQ + g, n & 1)) return false;
                fence_proxy_async();
                tc_fence_after();
            }
            const uint32_t tS = tmem + g * 256;
            const uint64_t qd = qd0 + g * (L::NB * L::kQBox / 16);
            if (elected()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma(tS, qd + (k / 4) * (L::kQBox / 16) + (k % 4) * 2,
                           kd + (k / 4) * (L::kKVBox / 16) + (k % 4) * 2, idesc_s, k > 0);
                tc_commit(bar(L::kBarS + g));
                if (i == te - 1) tc_commit(bar(L::kBarQE + g));
            }
            __syncwarp();
            return true;
        };
        auto kd = [&](int s) { return kd0 + (uint64_t)(s * (L::kTileBytes / 16)); };
        auto vd = [&](int s) { return vd0 + (uint64_t)(s * (L::kTileBytes / 16)); };
        auto ready = [&](int full, int s, int tile) {
            return poll(full + s, (tile / ST) & 1);
        };
        int n = -1;  // the job's number
        for (int r = 0; ok; ++r) {
            const int js = r % kJobs;
            if (!poll(L::kBarJF + js, (r / kJobs) & 1)) break;
            const Job *R = ring + js;
            const int te[kG] = {all(R->h[0].te), all(R->h[1].te)}, nt = all(R->nt), valid = all(R->valid);
            const bool pair = all(R->pair);
            one_arrive(bar(L::kBarJE + js));
            if (valid == kNoJob) break;
            if (valid == kLists) {
                after_previous();
                continue;
            }
            ++n;
            // a Q tile without tiles in this job is released at once
#pragma unroll
            for (int g = 0; g < kG; ++g)
                if (ok && te[g] == 0) {
                    ok = poll(L::kBarQ + g, n & 1);
                    if (ok) one_arrive(bar(L::kBarQE + g));
                }
            if (pair) {  // each Q tile has its own keys
                for (int i = 0; ok && i <= nt; ++i) {
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        const int tk = t + 2 * i + g, tv = tk - 2, sk = tk % ST, sv = (tv + 2 * ST) % ST;
                        if (ok && i > 0) {
                            ok = ready(L::kBarVF, sv, tv) && pv(g, i - 1, nt, vd(sv));
                            if (ok) one_commit(bar(L::kBarVE + sv));
                        }
                        if (ok && i < nt) {
                            ok = ready(L::kBarKF, sk, tk);
                            tc_fence_after();
                            if (ok) ok = qk(g, i, nt, kd(sk), n);
                            if (ok) one_commit(bar(L::kBarKE + sk));
                        }
                    }
                }
            } else {
                for (int i = 0; ok && i <= nt; ++i) {
                    const int tk = t + i, sk = tk % ST, sv = (sk + ST - 1) % ST;
                    const uint64_t kdi = kd(sk), vdi = vd(sv);
                    if (i < nt) {
                        ok = ready(L::kBarKF, sk, tk);
                        tc_fence_after();
                    }
                    if (ok && i > 0) ok = ready(L::kBarVF, sv, tk - 1);
#pragma unroll
                    for (int g = 0; g < kG; ++g) {
                        if (ok && i > 0 && i <= te[g]) ok = pv(g, i - 1, te[g], vdi);
                        if (ok && i < nt && i < te[g]) ok = qk(g, i, te[g], kdi, n);
                    }
                    if (!ok) break;
                    if (i < nt) one_commit(bar(L::kBarKE + sk));
                    if (i > 0) one_commit(bar(L::kBarVE + sv));
                }
            }
            t += pair ? 2 * nt : nt;
#pragma unroll
            for (int g = 0; g < kG; ++g) gt[g] += te[g];
        }
        one_commit(bar(L::kBarDrain));
        drain_bar(bar(L::kBarDrain), 0, ca.wait_limit);
        __syncwarp();
    } else {
        // ================= softmax (warps 2..9) =================
        const int g = (warp - 2) >> 2, quarter = warp & 3;
        const int trow = quarter * 32 + lane;  // row inside the Q tile
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_off + g * 256, tO = tS + 128;
        const uint32_t sQg = sQ + g * L::NB * L::kQBox;
        const uint32_t stg = base + L::kStage + (uint32_t)(warp - 2) * 4096u;
        const int S = a.km1 + 1;
        // what the Q tile's warps need of a job
        struct Mine {
            Half h;
            int valid, own, key_end, lo, pdelta, whole, slot, tiles;
        };
        // one inline look first: the bounded wait is a call
        auto wait = [&](int b, int parity) -> bool {
            return __all_sync(0xffffffffu, mbar_poll(bar(b), parity) || wait_bar(bar(b), parity, ctl));
        };
        // this thread's row of a job: row << 5 | slot
        auto entry_of = [&](const Mine &J) -> int {
            if (trow >= J.h.nrows) return -1;
            if (J.own) return (J.h.rbase + trow) << 5 | a.km1;
            // (two sequences that claim the same rows, from offsets that decrease,
            // spoil one another's lists: such an entry is no row)
            const int e = a.list[J.h.rbase + trow];
            return (unsigned)((e >> 5) - J.h.rlo) < (unsigned)J.h.rn && (e & 31) < a.km1 ? e : -1;
        };
        auto q_row = [&](int hk, int entry) -> size_t {
            const int row = entry >> 5;
            return (size_t)(row / a.G) * a.Hq + hk * a.G + row % a.G;
        };
        // the warp's 32 query rows into shared memory; zeros where there is no row
        auto gather = [&](int hk, int entry) {
            const unsigned long long mine =
                entry >= 0 ? reinterpret_cast<unsigned long long>(a.q + q_row(hk, entry) * D) : 0ull;
            const int ch = lane & 7;
#pragma unroll
            for (int it = 0; it < 8; ++it) {
                const int r = it * 4 + (lane >> 3);
                const unsigned long long p = __shfl_sync(0xffffffffu, mine, r);
                const __nv_bfloat16 *src = reinterpret_cast<const __nv_bfloat16 *>(p) + ch * 8;
                const uint32_t dst =
                    sQg + (uint32_t)(quarter * 32 + r) * 128 + ((uint32_t)(ch ^ (r & 7)) << 4);
#pragma unroll
                for (int x = 0; x < L::NB; ++x)
                    cp_async16(dst + x * L::kQBox, p ? (const void *)(src + x * 64) : (const void *)a.q,
                               p != 0);
            }
            cp_async_arrive_noinc(bar(L::kBarQ + g));
        };
        int r = 0;  // descriptors so far
        auto take = [&](Mine &J) -> bool {
            for (;;) {
                const int js = r % kJobs;
                if (!wait(L::kBarJF + js, (r / kJobs) & 1)) return false;
                const Job &R = ring[js];
                J.h = R.h[g];
                J.valid = R.valid;
                J.own = R.own;
                J.key_end = R.key_end;
                J.lo = R.lo;
                J.pdelta = R.pdelta;
                J.whole = R.whole;
                J.slot = R.slot;
                J.tiles = R.pair ? 2 * R.nt : R.nt;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kBarJE + js));
                ++r;
                if (DENSE || J.valid != kLists) return true;
                after_previous();
            }
        };
        int gt = 0, gj = 0, t = 0, n = 0;
        Mine J;
        bool ok = take(J);
        int entry = -1;
        if (ok && J.valid) {
            entry = entry_of(J);
            gather(J.h.hk, entry);
        }
        while (ok && J.valid) {
            const int ntile = J.h.te;
            // own blocks: positions that this row sees, [lo, hi]; a list's rows see
            // their block whole
            int lo = 0, hi = 0x7fffffff, lo_max = 0, hi_min = 0x7fffffff;
            if (J.own) {
                hi = SPANS && J.own == kFull ? J.key_end - 1 : (entry >> 5) / a.G + J.pdelta;
                if (!DENSE) lo = hi / a.c.bs * a.c.bs;
                // over the Q tile's rows: consecutive, so the first's and the last's
                hi_min = SPANS && J.own == kFull ? hi : J.h.rbase / a.G + J.pdelta;
                if (!DENSE)
                    lo_max = ((J.h.rbase + J.h.nrows - 1) / a.G + J.pdelta) / a.c.bs * a.c.bs;
            }
            float m_run = -INFINITY, l_run = 0.f;
            const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
            for (int j = 0; j < ntile; ++j) {
                if (!wait(L::kBarS + g, (gt + j) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int key0 = J.h.key0 + (J.lo + j) * N;
                const bool mask_hi = key0 + N - 1 > hi_min, mask_lo = key0 < lo_max;
#pragma unroll 1
                for (int h2 = 0; h2 < N / 64; ++h2) {
                    uint32_t sr[2][32];
                    tc_ld32(tS + 64 * h2, sr[0]);
                    tc_ld32(tS + 64 * h2 + 32, sr[1]);
                    tc_wait_ld();
                    if (mask_hi) {
                        const int top = hi - key0 - 64 * h2;  // last column that the row sees
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (c > top) sr[c >> 5][c & 31] = 0xff800000u;
                    }
                    if (!DENSE && mask_lo) {
                        const int bottom = lo - key0 - 64 * h2;
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            if (c < bottom) sr[c >> 5][c & 31] = 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int c = 0; c < 64; c += 2)
                        mx[(c >> 1) & 3] = fmax3(mx[(c >> 1) & 3], __uint_as_float(sr[c >> 5][c & 31]),
                                                 __uint_as_float(sr[c >> 5][(c & 31) + 1]));
                    const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale_log2;
                    const bool raise = mt > m_run + 8.f;
                    const float m_new = raise ? ceilf(mt) : m_run;
                    if (__any_sync(0xffffffffu, raise && (j > 0 || h2 > 0))) {
                        const float alpha = raise ? pow2_whole(m_run - m_new) : 1.f;
                        if (j > 0) {
#pragma unroll
                            for (int c0 = 0; c0 < D; c0 += 16) {
                                uint32_t o[16];
                                tc_ld16(tO + c0, o);
                                tc_wait_ld();
#pragma unroll
                                for (int c = 0; c < 16; ++c)
                                    o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                                tc_st16(tO + c0, o);
                            }
                        }
                        if (h2 > 0) {
                            // the first half's P was made with the old offset: rounded again,
                            // but by a power of two, so exact unless it underflows
                            tc_wait_st();
#pragma unroll
                            for (int c0 = 0; c0 < 32; c0 += 16) {
                                uint32_t pw[16];
                                tc_ld16(tS + c0, pw);
                                tc_wait_ld();
#pragma unroll
                                for (int c = 0; c < 16; ++c) {
                                    const float2 f =
                                        __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&pw[c]));
                                    __nv_bfloat162 bb = __floats2bfloat162_rn(f.x * alpha, f.y * alpha);
                                    pw[c] = *reinterpret_cast<uint32_t *>(&bb);
                                }
                                tc_st16(tS + c0, pw);
                            }
                        }
                    }
                    if (raise) {
                        l_run *= pow2_whole(m_run - m_new);
                        m_run = m_new;
                    }
                    const float mu = m_run == -INFINITY ? 0.f : m_run;
                    const float2 nmu2 = make_float2(-mu, -mu);
                    float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float2 x = ffma2(make_float2(__uint_as_float(sr[(2 * c) >> 5][(2 * c) & 31]),
                                                           __uint_as_float(sr[(2 * c + 1) >> 5][(2 * c + 1) & 31])),
                                               sc2, nmu2);
                        const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                        ls[c & 1] = fadd2(ls[c & 1], pp);
                        __nv_bfloat162 bb = __floats2bfloat162_rn(pp.x, pp.y);
                        pk[c] = *reinterpret_cast<uint32_t *>(&bb);
                    }
                    tc_st32(tS + 32 * h2, pk);
                    l_run += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
                }
                if (J.own && key0 + N > J.key_end) {
                    // keys that no row sees: zeros in V (both Q tiles' warps write
                    // the same zeros, each before its own product)
                    const int tv = t + j;
                    if (!__all_sync(0xffffffffu, wait_bar(bar(L::kBarVF + tv % ST), (tv / ST) & 1, ctl))) {
                        ok = false;
                        break;
                    }
                    const int nv = J.key_end - key0;
                    const int rows = N - nv, per = rows * 8;
                    for (int i = quarter * 32 + lane; i < per * L::NB; i += kM)
                        st_shared_v4(sV + (tv % ST) * L::kTileBytes + (i / per) * L::kKVBox + nv * 128 +
                                         (i % per) * 16,
                                     0, 0, 0, 0);
                    fence_proxy_async();
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::kBarP + g));
            }
            if (!ok) break;
            gt += ntile;
            t += J.tiles;
            // the next job's rows, as soon as this job's S MMAs have read Q
            Mine NJ;
            if (!take(NJ)) {
                ok = false;
                break;
            }
            int next_entry = -1;
            if (NJ.valid) {
                next_entry = entry_of(NJ);
                if (!wait(L::kBarQE + g, n & 1)) {
                    ok = false;
                    break;
                }
                gather(NJ.h.hk, next_entry);
            }
            // ---------------- results ----------------
            const bool bad = bad_job[n % kBadSlots] == n + 1;
            if (bad && lane == 0) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
            if (ntile > 0) {
                if (!wait(L::kBarPV + g, gj & 1)) {
                    ok = false;
                    break;
                }
                ++gj;
                tc_fence_after();
                // (a block whose scores are all -inf has weight 0 beside others)
                const float inv = !DENSE && l_run == 0.f ? 0.f : 1.f / l_run;
                const float lse2 = m_run + __log2f(l_run);
                if constexpr (!DENSE) {
                    // fp16 with a scale, 64 columns a pass, straight from the row's
                    // thread in whole 32-byte sectors (through shared memory, for whole
                    // lines, this took three times the instructions, and a tenth of the
                    // kernel)
                    const size_t at = ((size_t)J.h.hk * a.c.total * a.G + (max(entry, 0) >> 5)) * S +
                                      (max(entry, 0) & 31);
                    __half *dst = a.part_h + at * D;
                    float back[2] = {0.f, 0.f};
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 64) {
                        uint32_t o[2][32];
                        tc_ld32(tO + c0, o[0]);
                        tc_ld32(tO + c0 + 32, o[1]);
                        tc_wait_ld();
                        float mx[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            mx[c & 3] = fmaxf(mx[c & 3], fabsf(__uint_as_float(o[c >> 5][c & 31])));
                        // the largest value into [2^14, 2^15)
                        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * inv;
                        const int ex = min(max((__float_as_int(top) >> 23) & 255, 15), 254);
                        const float f = inv * __int_as_float((268 - ex) << 23);
                        back[c0 / 64] = __int_as_float((ex - 14) << 23);
                        const float2 f2 = make_float2(f, f), zero = make_float2(0.f, 0.f);
                        uint32_t w[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            const float2 x = ffma2(
                                make_float2(__uint_as_float(o[(2 * c) >> 5][(2 * c) & 31]),
                                            __uint_as_float(o[(2 * c + 1) >> 5][(2 * c + 1) & 31])),
                                f2, zero);
                            __half2 hh = __floats2half2_rn(x.x, x.y);
                            w[c] = *reinterpret_cast<uint32_t *>(&hh);
                        }
                        if (entry >= 0) {
#pragma unroll
                            for (int c = 0; c < 32; c += 8)
                                asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(
                                                 dst + c0 + 2 * c),
                                             "r"(w[c]), "r"(w[c + 1]), "r"(w[c + 2]), "r"(w[c + 3]),
                                             "r"(w[c + 4]), "r"(w[c + 5]), "r"(w[c + 6]), "r"(w[c + 7])
                                             : "memory");
                        }
                    }
                    if (entry >= 0)
                        a.part_s[at] = make_float4(lse2, back[0], back[1], bad ? 0.f : 1.f);
                } else if (!SPANS && J.whole) {
                    // the bf16 result, 64 columns a pass, 128 bytes of each row
                    const size_t at = q_row(J.h.hk, max(entry, 0));
                    const unsigned long long mine =
                        entry >= 0 ? reinterpret_cast<unsigned long long>(a.out + at * D) : 0ull;
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 64) {
                        uint32_t o[2][32];
                        tc_ld32(tO + c0, o[0]);
                        tc_ld32(tO + c0 + 32, o[1]);
                        tc_wait_ld();
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch) {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int c = ch * 8 + 2 * e;
                                __nv_bfloat162 bb = __floats2bfloat162_rn(
                                    __uint_as_float(o[c >> 5][c & 31]) * inv,
                                    __uint_as_float(o[(c + 1) >> 5][(c + 1) & 31]) * inv);
                                w[e] = bad ? 0u : *reinterpret_cast<uint32_t *>(&bb);
                            }
                            st_shared_v4(stg + lane * 128 + ((uint32_t)(ch ^ (lane & 7)) << 4), w[0], w[1],
                                         w[2], w[3]);
                        }
                        __syncwarp();
#pragma unroll
                        for (int it = 0; it < 8; ++it) {
                            const int r = it * 4 + (lane >> 3), ch = lane & 7;
                            const unsigned long long d = __shfl_sync(0xffffffffu, mine, r);
                            const uint4 val = ld_shared_v4(stg + r * 128 + ((uint32_t)(ch ^ (r & 7)) << 4));
                            if (d)
                                *reinterpret_cast<uint4 *>(reinterpret_cast<__nv_bfloat16 *>(d) + c0 + ch * 8) = val;
                        }
                        __syncwarp();
                    }
                    if (entry >= 0) a.lse[at] = bad ? -INFINITY : lse2 * 0.69314718055994530942f;
                } else {
                    // fp32 partial sums, 32 columns a pass
                    float *prow = a.part_o + ((size_t)J.slot * kJobRows + g * kM + quarter * 32) * D;
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tc_ld32(tO + c0, o);
                        tc_wait_ld();
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch)
                            st_shared_v4(stg + lane * 128 + ((uint32_t)(ch ^ (lane & 7)) << 4), o[4 * ch],
                                         o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]);
                        __syncwarp();
#pragma unroll
                        for (int it = 0; it < 8; ++it) {
                            const int r = it * 4 + (lane >> 3), ch = lane & 7;
                            const uint4 val = ld_shared_v4(stg + r * 128 + ((uint32_t)(ch ^ (r & 7)) << 4));
                            if (quarter * 32 + r < J.h.nrows)
                                *reinterpret_cast<uint4 *>(prow + (size_t)r * D + c0 + ch * 4) = val;
                        }
                        __syncwarp();
                    }
                    if (entry >= 0)
                        a.part_ml[(size_t)J.slot * kJobRows + g * kM + trow] = make_float2(m_run, bad ? -1.f : l_run);
                }
                // O may be overwritten
                tc_fence_before();
            } else if (DENSE && entry >= 0) {
                // rows that see nothing of this part
                a.part_ml[(size_t)J.slot * kJobRows + g * kM + trow] = make_float2(-INFINITY, bad ? -1.f : 0.f);
            }
            ++n;
            J = NJ;
            entry = next_entry;
        }
        cp_async_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
    }
}

// ----------------------------------------------------------------------------
// row tiles, list offsets and jobs (one CTA), and the lists
// ----------------------------------------------------------------------------
// The plan goes by the lists in use, not by the page table's width: a chunk of 600 beside
// 64 steps takes 73 us in tables of 256 to 8192 blocks (192 to 7700 when every list of
// the table was walked).  1 ns for a list in use where they are many (16.8 M of 512
// sequences that share a long cache: 15.8 ms for the whole call).
constexpr int kPlanThreads = 1024, kPlanLists = 4;

// inclusive sums over the CTA's threads, N at a time
template <int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long (*warps)[kPlanThreads / 32],
                                           long long (&total)[N]) {
    static_assert(kPlanThreads == 1024, "a warp scans the warps' sums");
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
        long long s = warps[i][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        total[i] = __shfl_sync(0xffffffffu, s, 31);
        const long long before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
        v[i] += warp > 0 ? before : 0;
    }
}

template <int N>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(Attn a) {
    __shared__ long long warps[2][kPlanThreads / 32];
    __shared__ int s_off[kPlanThreads + 1];  // `off`, where that is no longer
    let_next();
    after_previous();
    const int tid = threadIdx.x;
    // 256-row tiles of each sequence (all blocks), or its lists in use: those of the
    // blocks before its last, whatever the page table's width; refused ones have none,
    // and clear rows
    long long run = 0;
    int *off = a.dense ? a.own_off : a.used_off;
    const long long most = a.dense ? a.w_cap : (long long)a.c.num_seqs * a.n_max * a.c.Hkv;
    for (int b0 = 0; b0 < a.c.num_seqs; b0 += kPlanThreads) {
        const int b = b0 + tid;
        Seq s;
        const int state = b < a.c.num_seqs ? a.c.seq(b, s) : (int)kSeqEmpty;
        if (state == kSeqBad) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
        if (__syncthreads_or(state == kSeqBad))
            for (int r = b0; r < min(b0 + kPlanThreads, a.c.num_seqs); ++r) {
                Seq x;
                if (a.c.seq(r, x) == kSeqBad) clear_refused(a, x, 0, a.Hq, tid, kPlanThreads);
            }
        long long inc[1] = {0}, total[1];
        if (state == kSeqOk)
            inc[0] = a.dense ? ((long long)s.n * a.G + kJobRows - 1) / kJobRows
                             : (long long)((s.len - 1) / a.c.bs) * a.c.Hkv;
        block_scan(inc, warps, total);
        if (b < a.c.num_seqs) {
            off[b + 1] = (int)min(run + inc[0], most);
            if (b < kPlanThreads) s_off[b + 1] = off[b + 1];
        }
        run += total[0];
    }
    if (tid == 0) off[0] = s_off[0] = 0;
    __threadfence_block();
    __syncthreads();
    if (a.dense) {
        const int tiles = (int)min(run, most);
        run = 0;
        for (int w0 = 0; w0 < tiles; w0 += kPlanThreads) {
            const int w = w0 + tid;
            long long inc[1] = {0}, total[1];
            if (w < tiles) {
                const int b = seq_of_tile(a, w);
                Seq s;
                a.c.seq(b, s);
                Job J;
                own_job<N>(a, s, b, 0, w - a.own_off[b], J);
                inc[0] = (long long)J.nt * a.c.Hkv;
            }
            block_scan(inc, warps, total);
            if (w < tiles) a.unit_off[w + 1] = run + inc[0];
            run += total[0];
        }
        if (tid == 0) a.unit_off[0] = 0;
        return;
    }
    if (tid == 0) a.n_jobs[2] = 0;
    if (a.km1 == 0) return;
    // offsets of the lists, a job for every 256 rows of one, and the last rows: a
    // job where they are more than 128, else half of one
    const int lists = (int)run;
    const int *before = a.c.num_seqs <= kPlanThreads ? s_off : off;
    long long row = 0, job = 0, half = 0;
    for (int i0 = 0; i0 < lists;) {
        // consecutive lists a thread, consecutive threads: loads and stores of whole lines
        const int per = min(kPlanLists, (lists - i0 + kPlanThreads - 1) / kPlanThreads);
        const int i = i0 + tid * per, end = min(i + per, lists);
        i0 += kPlanThreads * per;
        int at[kPlanLists], n[kPlanLists];
        long long inc[2] = {0, 0}, total[2];  // rows; jobs << 32 | halves (both stay below 2^31)
        if (i < lists) {
            int b = 0, hi = a.c.num_seqs - 1;
            while (b < hi) {
                const int mid = (b + hi + 1) >> 1;
                if (before[mid] <= i) b = mid; else hi = mid - 1;
            }
#pragma unroll
            for (int k = 0; k < kPlanLists; ++k)
                if (i + k < end) {
                    while (before[b + 1] <= i + k) ++b;
                    at[k] = b * a.n_max * a.c.Hkv + i + k - before[b];
                    n[k] = a.counts[at[k]];
                }
#pragma unroll
            for (int k = 0; k < kPlanLists; ++k)
                if (i + k < end) {
                    const int rest = n[k] % kJobRows;
                    inc[0] += n[k];
                    inc[1] += (long long)(n[k] / kJobRows + (rest > kM)) << 32 | (rest > 0 && rest <= kM);
                }
        }
        const long long mine[2] = {inc[0], inc[1]};
        block_scan(inc, warps, total);
        long long r = row + inc[0] - mine[0];
        long long j = job + ((inc[1] - mine[1]) >> 32), h = half + ((inc[1] - mine[1]) & 0xffffffffll);
#pragma unroll
        for (int k = 0; k < kPlanLists; ++k)
            if (i + k < end) {
                a.list_off[at[k]] = (int)min(r, a.list_cap);
                int s = 0;
                for (; n[k] - s > kM; s += kJobRows, ++j)
                    if (j < a.job_cap) a.jobs[j] = make_int2(at[k], s);
                if (s < n[k]) {
                    if (h < a.job_cap) a.halves[h] = make_int2(at[k], s);
                    ++h;
                }
                r += n[k];
            }
        row += total[0];
        job += total[1] >> 32;
        half += total[1] & 0xffffffffll;
    }
    // (more rows than the tensors hold: only from offsets that overlap, refused ones among them)
    if (tid == 0) {
        a.n_jobs[0] = (int)min(job, a.job_cap);
        a.n_jobs[1] = (int)min(half, a.job_cap);
    }
}

// The rows into the lists of the blocks that they selected; a row's slots are
// its past blocks in ascending order.  Latency: 8 us for 262144 entries (the plan 6 us).
constexpr int kScatterThreads = 1024;

__global__ void __launch_bounds__(kScatterThreads) scatter_kernel(Attn a) {
    let_next();
    after_previous();
    const int hk = blockIdx.y;
    const long long n = (long long)a.c.total * a.G * a.km1;
    for (long long i = (long long)blockIdx.x * kScatterThreads + threadIdx.x; i < n;
         i += (long long)gridDim.x * kScatterThreads) {
        const int row = (int)(i / a.km1), slot = (int)(i - (long long)row * a.km1);
        const int2 c = a.sel[hk * n + i];
        if (a.tok[row / a.G] == 0 || c.x < 0) continue;
        const long long at = (long long)a.list_off[c.x] + c.y;
        if (at < a.list_cap) a.list[at] = row << 5 | slot;
    }
}

// ----------------------------------------------------------------------------
// merge
// ----------------------------------------------------------------------------
// A row's slots (its past blocks and its own), weighted by their sums, the
// weights taken relative to a running maximum: D / 16 lanes a row, 32 bytes of
// each slot a lane, up to four slots in flight.  Bound: HBM and L2 (the partials),
// then the issue of instructions, so a lane does much per row and index
// arithmetic is kept to one division.  131072 rows of three slots of 128: 27 us,
// 5 TB/s of partials and results.
constexpr int kSlotThreads = 256;

template <int D>
__global__ void __launch_bounds__(kSlotThreads, 3) merge_slots_kernel(Attn a) {
    constexpr int GL = D / 16, U = 4, ROWS = kSlotThreads / GL;
    after_previous();
    const int hk = blockIdx.y, gl = threadIdx.x % GL, S = a.km1 + 1, G = a.G;
    const int nrows = a.c.total * G;
    const size_t base = (size_t)hk * nrows;
    for (int row = blockIdx.x * ROWS + threadIdx.x / GL; row < nrows; row += gridDim.x * ROWS) {
        const int t = row / G, pos1 = a.tok[t];
        if (pos1 == 0) continue;  // (refused ones are cleared by the plan)
        const size_t lin = base + row, p0 = lin * S;
        // slots, the own block's last
        const int n = min(a.km1, (pos1 - 1) / a.c.bs) + 1;
        bool bad = a.km1 > 0 && a.sel[lin * a.km1].x == kSelBad;
        float M = -INFINITY, W = 0.f, acc[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) acc[k] = 0.f;
        for (int s0 = 0; s0 < n; s0 += U) {
            float4 ps[U];
            uint4 h[U][2];
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s0 + j < n) {
                    const size_t p = p0 + (s0 + j < n - 1 ? s0 + j : a.km1);
                    ps[j] = a.part_s[p];
                    const uint4 *src = reinterpret_cast<const uint4 *>(a.part_h + p * D) + 2 * gl;
                    h[j][0] = __ldcs(src);
                    h[j][1] = __ldcs(src + 1);
                }
            float mx = M;
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s0 + j < n) mx = fmaxf(mx, ps[j].x);
            if (s0 > 0 && mx > M) {
                const float f = fast_exp2(M - mx);
                W *= f;
#pragma unroll
                for (int k = 0; k < 16; ++k) acc[k] *= f;
            }
            M = mx;
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int j = 0; j < U; ++j)
                if (s0 + j < n) {
                    bad |= ps[j].w == 0.f;
                    const float w = fast_exp2(ps[j].x - ref);
                    W += w;
                    const float f = w * (gl < 4 ? ps[j].y : ps[j].z);
                    const __half2 *h2 = reinterpret_cast<const __half2 *>(h[j]);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 v = __half22float2(h2[k]);
                        acc[2 * k] = fmaf(v.x, f, acc[2 * k]);
                        acc[2 * k + 1] = fmaf(v.y, f, acc[2 * k + 1]);
                    }
                }
        }
        const float inv = 1.f / W;
        uint4 o[2];
        __nv_bfloat162 *o2 = reinterpret_cast<__nv_bfloat162 *>(o);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            o2[k] = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
        if (bad) o[0] = o[1] = make_uint4(0, 0, 0, 0);
        const size_t at = (size_t)t * a.Hq + hk * G + (row - t * G);
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * D) + 2 * gl;
        dst[0] = o[0];
        dst[1] = o[1];
        if (gl == 0) a.lse[at] = bad ? -INFINITY : (M + log2f(W)) * 0.69314718055994530942f;
    }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------
template <int D, int N, bool DENSE, bool SPANS = false>
cudaError_t launch(const Attn &a, cudaStream_t st) {
    CUtensorMap mk, mv;
    const long long rows = (long long)a.c.num_pages * a.c.Hkv * a.c.ps;
    const int box = a.c.ps < N ? a.c.ps : N;
    if (!make_tma_rows(&mk, a.k, rows, D, box) || !make_tma_rows(&mv, a.v, rows, D, box))
        return cudaErrorInvalidValue;
    const int bytes = (int)Smem<D, N>::kRequest;
    // every warp role must be resident: refuse a build whose registers do not allow it
    static std::atomic<int> fits{0};
    if (fits.load(std::memory_order_relaxed) == 0) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, chunk_kernel<D, N, DENSE, SPANS>);
        if (e != cudaSuccess) return e;
        fits.store(fa.maxThreadsPerBlock >= kThreads ? 1 : -1, std::memory_order_relaxed);
    }
    if (fits.load(std::memory_order_relaxed) < 0) return cudaErrorInvalidConfiguration;
    cudaError_t rc = allow_smem<chunk_kernel<D, N, DENSE, SPANS>>(bytes);
    if (rc != cudaSuccess) return rc;
    ChunkArgs ca;
    ca.a = a;
    ca.psh = __builtin_ctz((unsigned)a.c.ps);
    ca.wait_limit = kDefaultWaitLimit;
    rc = launch_after(chunk_kernel<D, N, DENSE, SPANS>, a.ctas, kThreads, bytes, st, mk, mv, ca);
    note_launches(1);
    if (rc != cudaSuccess) return rc;
    if (SPANS) return cudaSuccess;
    if (DENSE) return launch_merge_runs(a, st);
    note_launches(1);
    constexpr int ROWS = kSlotThreads / (D / 16);
    const long long tiles = ((long long)a.c.total * a.G + ROWS - 1) / ROWS;
    const long long fill = (3 * a.ctas + a.c.Hkv - 1) / a.c.Hkv;
    const dim3 grid((unsigned)(tiles < fill ? tiles : fill), a.c.Hkv);
    return launch_after(merge_slots_kernel<D>, grid, kSlotThreads, 0, st, a);
}

// keys per tile: 128, or 64 where blocks are no multiple of 128
bool wide(const Attn &a) { return a.dense || a.c.bs % 128 == 0; }

}  // namespace

cudaError_t launch_plan(const Attn &a, bool after_gate, cudaStream_t st) {
    cudaError_t rc;
    const auto plan = wide(a) ? plan_kernel<128> : plan_kernel<64>;
    if (after_gate) {
        rc = launch_after(plan, 1, kPlanThreads, 0, st, a);
    } else {
        plan<<<1, kPlanThreads, 0, st>>>(a);
        rc = cudaGetLastError();
    }
    note_launches(1);
    if (rc != cudaSuccess || a.km1 == 0) return rc;
    note_launches(1);
    const long long most = (long long)a.c.total * a.G * a.km1;
    // few and large CTAs: the other SMs begin with their own blocks meanwhile
    const long long ctas = (most + 4 * kScatterThreads - 1) / (4 * kScatterThreads);
    const long long cap = (a.ctas / 3 + a.c.Hkv - 1) / a.c.Hkv;
    const dim3 grid((unsigned)(ctas < cap ? ctas : cap), a.c.Hkv);
    return launch_after(scatter_kernel, grid, kScatterThreads, 0, st, a);
}

cudaError_t launch_chunk(const Attn &a, cudaStream_t st) {
    if (a.dense) return a.D == 64 ? launch<64, 128, true>(a, st) : launch<128, 128, true>(a, st);
    if (wide(a)) return a.D == 64 ? launch<64, 128, false>(a, st) : launch<128, 128, false>(a, st);
    return a.D == 64 ? launch<64, 64, false>(a, st) : launch<128, 64, false>(a, st);
}

cudaError_t launch_chunk_spans(const Attn &a, cudaStream_t st) {
    return a.D == 64 ? launch<64, 128, true, true>(a, st) : launch<128, 128, true, true>(a, st);
}

}  // namespace paged
}  // namespace moba
