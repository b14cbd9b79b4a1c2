// moba_paged_rope.cu -- appending new tokens to a paged cache with the position
// rotation, and the norms of queries and keys, applied on the way.
//
// Pages: "When a MoBA reproduction will not run" (mhpq.cn/news/582794) section
// 3.3 (where positions enter) and "MOBA mixture of block attention for server-side
// long context" (hncyxsy.com/news/197418) section 3 (pooled block keys); the pages
// describe no paged cache.
//
// q and k of a new token are normalised over each head (where weights are given),
// rotated to the token's position and rounded once; q goes to q_out, k and v to the
// token's page.  k is then never in memory unrotated: q, k and v are read and written
// once, 4 bytes a value, from slices of one projection as they are.  A second launch
// pools the blocks that the tokens complete from the keys as stored, with the kernel and
// in the order of moba_paged_append, so that a pooled key is the same bits whichever
// call wrote its keys.
//
// Bound: HBM for chunks, latency for a step.  A warp takes one token and a run of its
// heads (q, then k, then v).  Measured (32 + 8 + 8 heads of 128, normalised): 16469 tokens in
// four chunks 72 us, 5.6 TB/s (the pages' rows of 256 bytes are scattered writes), and 16 for
// pooling 32 blocks of 512, 91 by the call; a step of 64 sequences of which one completes its
// block 10.8.  (Units of a third of a token 102 by the call; tokens in consecutive runs a warp 112; CTAs
// in waves 98; k and v first and q beside the pooling, in a launch of its own, 98.)
#include <cmath>

#include "moba_paged.cuh"
#include "moba_rope.cuh"

namespace moba {
namespace paged {
namespace {

using namespace rope;

constexpr int kWarps = 8;
constexpr int kUnroll = 4;  // heads of a lane in a step
constexpr int kCtas = 2;    // of an SM

struct WriteArgs {
    Cache c;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *qo, *kp, *vp;
    long long qs, ks, vs, qos;  // elements between tokens
    const void *wq, *wk;        // norm weights, or nullptr: not normalised
    const int *pos;             // or nullptr: the token's place in its sequence
    const double *freqs;
    int Hq, rot, psh;
    int chunk, splits;          // heads per unit, units per token
    int w32;                    // weights are fp32 (else bf16)
    float eps, mag;
    int *status;
    unsigned long long *ready, token;  // for the pooling (nullptr: none)
};

// A warp works through its units' steps, kUnroll heads of every lane each, of q, of k or
// of v, which come by bulk copies two steps ahead.
using StepRing = WarpRing<3, kUnroll * 1024>;  // 32 lanes * 16 values

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, kCtas) write_kernel(WriteArgs a) {
    constexpr int LH = D / 16;   // lanes per head: 16 values (8 pairs) each
    constexpr int HW = 32 / LH, STEP = HW * kUnroll;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ __align__(8) unsigned long long s_bar[kWarps][StepRing::kStages];
    __shared__ int s_abort;
    __shared__ unsigned long long s_turn[D / 2];
    __shared__ __align__(16) float s_w[2][D], s_c[kWarps][D / 2], s_s[kWarps][D / 2];
    after_previous();
    if (a.ready && blockIdx.x == 0 && threadIdx.x == 0) ptx::st_release(a.ready, a.token);
    let_next();
    load_turns(s_turn, a.freqs, a.rot / 2, threadIdx.x, 32 * kWarps);
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps) {
        const void *w = i < D ? a.wq : a.wk;
        if (w) s_w[i / D][i % D] = weight(w, a.w32, i % D);
    }
    // refused sequences are reported, rows or not
    for (int b = blockIdx.x * 32 * kWarps + threadIdx.x; b < a.c.num_seqs; b += gridDim.x * 32 * kWarps) {
        Seq s;
        if (a.c.seq_now(b, s) == kSeqBad) atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
    }
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w) StepRing::init(s_bar[w]);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, item = lane % LH, hsub = lane / LH;
    const int Hkv = a.c.Hkv, heads = a.Hq + 2 * Hkv, ps = a.c.ps;
    const bool turns = item < a.rot / 16;  // the other items are not rotated
    int va, vb;
    vectors<D, INTERLEAVED>(item, a.rot / 2, va, vb);
    const int warp = threadIdx.x >> 5;
    const unsigned units = (unsigned)a.c.total * a.splits, stride = gridDim.x * kWarps;
    auto token = [&](unsigned u) { return (int)(a.splits == 1 ? u : u / a.splits); };
    auto begin = [&](unsigned u) { return a.splits == 1 ? 0 : (int)(u % a.splits) * a.chunk; };
    // of the kinds q, k, v: their first head among all, and the first behind them
    auto base = [&](int kind) { return kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + Hkv; };
    auto limit = [&](int kind, int hi) { return min(hi, kind == 0 ? a.Hq : kind == 1 ? a.Hq + Hkv : heads); };
    auto kind_of = [&](int h) { return (h >= a.Hq) + (h >= a.Hq + Hkv); };
    ptx::Ctl ctl{&s_abort, a.status, kDefaultWaitLimit};
    StepRing ring(s_bar[warp], ptx::saddr(s_ring) + warp * StepRing::kBytes);
    unsigned u = blockIdx.x * kWarps + warp, nu = u;                      // the unit at hand, the one to be copied next
    int nh = begin(min(u, units - 1)), nhi = min(nh + a.chunk, heads);    // its heads that are left
    auto issue = [&] {
        if (nu >= units) return;
        const int t = token(nu), kind = kind_of(nh), n = min(STEP, limit(kind, nhi) - nh);
        const __nv_bfloat16 *row = kind == 0 ? a.q + t * a.qs : kind == 1 ? a.k + t * a.ks : a.v + t * a.vs;
        const void *const src[1] = {row + (size_t)(nh - base(kind)) * D};
        ring.fill(lane, src, (uint32_t)n * D * 2);
        nh += n;
        if (nh >= nhi && (nu += stride) < units) {
            nh = begin(nu);
            nhi = min(nh + a.chunk, heads);
        }
    };
#pragma unroll 1
    for (int i = 0; i < StepRing::kStages - 1; ++i) issue();
    bool ok = true;
    for (; ok && u < units; u += stride) {
        const int t = token(u), h0 = begin(u), h1 = min(h0 + a.chunk, heads);
        const int b = a.c.seq_of_row(t, lane);
        Seq s;
        // (rows of no sequence, or of a refused one, are left as they were)
        const bool live = a.c.seq_now(b, s) == kSeqOk && t >= s.row0 && t < s.row0 + s.n;
        const int p = live ? s.len - s.n + t - s.row0 : 0;  // the token's place
        __nv_bfloat16 *page_k = nullptr, *page_v = nullptr;
        if (live && h1 > a.Hq) {
            const int page = a.c.table[(size_t)b * a.c.max_pages + (p >> a.psh)];
            if ((unsigned)page < (unsigned)a.c.num_pages) {
                const size_t at = (((size_t)page * Hkv << a.psh) + (p & (ps - 1))) * D;
                page_k = a.kp + at;
                page_v = a.vp + at;
            } else if (lane == 0) {
                atomicCAS(a.status, 0, (int)MOBA_ERR_INVALID_ARG);
            }
        }
        float2 c[4], sn[4];
        if (h0 < a.Hq + Hkv) {
            warp_cos_sin(s_turn, a.rot / 2, lane, a.pos ? a.pos[t] : p, a.mag, 1.f, s_c[warp], s_s[warp]);
            if (turns) {
                load_eight(s_c[warp] + item * 8, c);
                load_eight(s_s[warp] + item * 8, sn);
            }
        }
#pragma unroll 1
        for (int hb = h0, n; hb < h1; hb += n) {
            issue();
            const uint32_t stage = ring.wait(ctl);
            ok = stage != 0;
            if (!ok) break;
            const int kind = kind_of(hb);
            n = min(STEP, limit(kind, h1) - hb);
            __nv_bfloat16 *dst = !live ? nullptr : kind == 0 ? a.qo + t * a.qos : kind == 1 ? page_k : page_v;
            const size_t step = kind == 0 ? (size_t)D : (size_t)D << a.psh;  // between heads of dst
            const bool norm = kind == 0 ? a.wq != nullptr : kind == 1 && a.wk != nullptr;
            const float *w = s_w[kind & 1];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int i = j * HW + hsub;
                if (j * HW >= n) break;  // (the warp alike)
                uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
                if (i < n) {
                    xa = ptx::ld_shared_v4(stage + i * D * 2 + 2 * va);
                    xb = ptx::ld_shared_v4(stage + i * D * 2 + 2 * vb);
                }
                if (kind < 2 && (norm || turns)) {  // (else copied as they are, NaN payloads too)
                    float2 fa[4], fb[4];
                    unpack(xa, fa);
                    unpack(xb, fb);
                    if (norm) {
                        float2 wa[4], wb[4];
                        load_eight(w + va, wa);
                        load_eight(w + vb, wb);
                        normalise<D>(fa, fb, wa, wb, a.eps);
                    }
                    if (turns) turn_pairs<INTERLEAVED>(fa, fb, c, sn);
                    xa = pack(fa);
                    xb = pack(fb);
                }
                if (dst && i < n) {
                    *reinterpret_cast<uint4 *>(dst + (hb + i - base(kind)) * step + va) = xa;
                    *reinterpret_cast<uint4 *>(dst + (hb + i - base(kind)) * step + vb) = xb;
                }
            }
            ring.release();
        }
    }
    ring.drain();
}

template <int D>
cudaError_t launch_write(const WriteArgs &a, bool interleaved, cudaStream_t st) {
    const long long units = (long long)a.c.total * a.splits;
    const long long want = (units + kWarps - 1) / kWarps, cap = (long long)sm_count() * kCtas;
    const int grid = (int)(want < cap ? want : cap);
    constexpr int bytes = kWarps * StepRing::kBytes;
    const cudaError_t rc = interleaved ? allow_smem<write_kernel<D, true>>(bytes) : allow_smem<write_kernel<D, false>>(bytes);
    if (rc != cudaSuccess) return rc;
    note_launches(1);
    return interleaved ? launch_after(write_kernel<D, true>, dim3(grid), dim3(32 * kWarps), bytes, st, a)
                       : launch_after(write_kernel<D, false>, dim3(grid), dim3(32 * kWarps), bytes, st, a);
}

}  // namespace
}  // namespace paged
}  // namespace moba

using namespace moba;
using namespace moba::paged;

MOBA_EXPORT int moba_paged_append_rope(const void *q, const void *k, const void *v, void *q_out, void *k_pages,
                                       void *v_pages, float *kbar_pages, const int32_t *page_table,
                                       const int32_t *cu_new, const int32_t *cache_lens, const int32_t *positions,
                                       const double *freqs, const void *q_weight, const void *k_weight,
                                       int weight_bits, float eps, int num_seqs, int total, int max_new, int Hq,
                                       int Hkv, int D, int rot_dim, int interleaved, float magnitude,
                                       long long q_stride, long long k_stride, long long v_stride,
                                       long long q_out_stride, int num_pages, int page_size, int max_pages,
                                       int block_size, const moba_options_t *options, void *stream) {
    int pooling = MOBA_POOL_MEAN;
    if (options) {
        if (options->pooling != MOBA_POOL_MEAN && options->pooling != MOBA_POOL_MAX) return MOBA_ERR_INVALID_ARG;
        pooling = options->pooling;
    }
    WriteArgs a = {};
    int rc = make_cache(&a.c, k_pages, v_pages, kbar_pages, page_table, cu_new, cache_lens, num_seqs, total, max_new,
                        Hkv, D, num_pages, page_size, max_pages, block_size);
    if (rc != MOBA_OK) return rc;
    if (Hq < 1 || !freqs || (reinterpret_cast<uintptr_t>(freqs) & 7) || (reinterpret_cast<uintptr_t>(positions) & 3))
        return MOBA_ERR_INVALID_ARG;
    if (Hq > 65535) return MOBA_ERR_UNSUPPORTED;
    if (rot_dim < 16 || rot_dim > D || rot_dim % 16 != 0) return MOBA_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || !std::isfinite(magnitude)) return MOBA_ERR_INVALID_ARG;
    if (q_weight || k_weight) {
        if (weight_bits != 16 && weight_bits != 32) return MOBA_ERR_INVALID_ARG;
        if (!(eps >= 1e-12f) || !std::isfinite(eps)) return MOBA_ERR_INVALID_ARG;
        if ((reinterpret_cast<uintptr_t>(q_weight) | reinterpret_cast<uintptr_t>(k_weight)) & (weight_bits / 8 - 1))
            return MOBA_ERR_INVALID_ARG;
    }
    rc = check_rows(q, Hq, D, total, &q_stride);
    if (rc == MOBA_OK) rc = check_rows(k, Hkv, D, total, &k_stride);
    if (rc == MOBA_OK) rc = check_rows(v, Hkv, D, total, &v_stride);
    if (rc == MOBA_OK) rc = check_rows(q_out, Hq, D, total, &q_out_stride);
    if (rc != MOBA_OK) return rc;
    // q_out may be q (in place), and overlaps nothing else that is read
    const long long wq = 2ll * Hq * D, wk = 2ll * Hkv * D;
    if ((q != q_out || q_stride != q_out_stride) &&
        overlaps(q, 2 * q_stride, wq, q_out, 2 * q_out_stride, wq, total))
        return MOBA_ERR_INVALID_ARG;
    if (overlaps(k, 2 * k_stride, wk, q_out, 2 * q_out_stride, wq, total) ||
        overlaps(v, 2 * v_stride, wk, q_out, 2 * q_out_stride, wq, total))
        return MOBA_ERR_INVALID_ARG;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.v = static_cast<const __nv_bfloat16 *>(v);
    a.qo = static_cast<__nv_bfloat16 *>(q_out);
    a.kp = static_cast<__nv_bfloat16 *>(k_pages);
    a.vp = static_cast<__nv_bfloat16 *>(v_pages);
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.qos = q_out_stride;
    a.wq = q_weight;
    a.wk = k_weight;
    a.pos = positions;
    a.freqs = freqs;
    a.Hq = Hq;
    a.rot = rot_dim;
    a.psh = __builtin_ctz((unsigned)page_size);
    a.w32 = weight_bits == 32;
    a.eps = eps;
    a.mag = magnitude;
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    AppendArgs pool;
    if (kbar_pages) {
        rc = make_pool(&pool, a.c, k_pages, kbar_pages, a.status);
        if (rc != MOBA_OK) return rc;
        a.ready = pool.ready;
        a.token = pool.token;
    }
    split_heads(Hq + 2 * Hkv, total, D, kUnroll, &a.chunk, &a.splits);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = D == 64 ? launch_write<64>(a, interleaved != 0, st) : launch_write<128>(a, interleaved != 0, st);
    if (e == cudaSuccess && kbar_pages) e = launch_pool(pool, D, pooling == MOBA_POOL_MAX, st);
    return cuda_result(e);
}
