// moba_qk_norm.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and their gradient.
//
// Pages: "When a MoBA reproduction will not run" (mhpq.cn/news/582794) section
// 3.3 asks where positions enter MoBA; here they enter before the gate, and so do the
// norms of models that bound their logits by normalising q and k.
//
// For a head x of D values with weights w:  r = 1 / sqrt(mean x^2 + eps),
//   y = R (x r w), R the rotation of moba_rope.
// Gradient, with g = R^T dy and n = x r:
//   dx = r (g w - n mean(g w n)),  dw = sum over tokens and heads of g n.
// Everything between the loads and the one rounding of the result is fp32; r and n are
// made again from x in the gradient, which costs nothing where x has to be read anyway.
//
// Bound: HBM (4 bytes a value, 6 in the gradient).  A lane has 16 values of a head, eight
// pairs, so that the norm is three shuffles; the phases of a token are made once by the
// warp's lanes; arithmetic is on pairs; operands come by bulk copies into a ring of stages for
// each warp, two steps ahead.  Measured: 32768 tokens of 64 heads of 128 160 us, 6.7 TB/s, 0.99 of
// the copy rate (from memory to registers 170; 15085 of 40 heads of 64 29 and 38); the gradient
// of 32764 tokens of 32 heads, half of each rotated, 125 us in its kernel, 6.4 TB/s, 130 by the
// call with the weights' sums.  (The gradient from memory to registers took 144: its 16
// warps an SM waited for loads half of the time; with the phases made by every lane for
// itself and 64-bit unit numbers 170.)
#include <algorithm>
#include <cmath>

#include "moba.h"
#include "moba_paged.cuh"
#include "moba_rope.cuh"

namespace moba {
namespace qk_norm {

using namespace rope;

constexpr int kWarps = 8;
constexpr int kUnroll = 4, kBwdUnroll = 2;  // heads of a lane in a step
constexpr int kFwdCtas = 2, kBwdCtas = 2;   // of an SM at a time
// CTAs come in waves, so that SMs which get through more (they differ by their distance from
// the memory) take more: a wave's start costs a microsecond or two, and in the gradient a row
// of sums for each of its CTAs.  The forward's, of at least so many steps a warp (one wave, four and
// eight at most: 32768 tokens of 64 heads of 128 183, 168, 162 us, 59022 of 40 of 64 110, 100, 97; 15085
// of these, eight steps, 29 with one and 33 with four).  The gradient's are four, of as many at least, or
// one (one, three, four and six: 32764 tokens of 40 heads of 128 182, 171, 167, 167, of 32 140, 132, 133,
// 137; 15085 of 40 of 64, 15 steps in all, 47 with one and 51 with three).
constexpr int kFwdWaves = 8, kWaveSteps = 5, kBwdWaves = 4, kBwdWaveSteps = 10;

struct Side {                   // q or k
    const __nv_bfloat16 *x, *dy;  // dy: gradient only
    __nv_bfloat16 *out;
    const void *w;
    long long xs, ds, os;       // elements between tokens
    int heads;
    int chunk, splits;          // gradient: heads per unit, units per token
};
struct Args {
    Side q, k;
    const int32_t *pos;
    const double *freqs;
    float *part;                // gradient: [CTAs][D] sums of the weights'
    int q_ctas;                 // gradient: CTAs of q, before those of k
    int tokens, rot;
    int chunk, splits;          // heads per unit, units per token
    int w32;                    // weights are fp32 (else bf16)
    int *status;
    bool wide;                  // every head of the results is aligned to 32 bytes
    float eps, mag;
};

// A warp works through its units' steps, kUnroll heads of every lane each, of q or of k,
// which come by bulk copies two steps ahead.
using FwdRing = WarpRing<3, kUnroll * 1024>;  // 32 lanes * 16 values

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, kFwdCtas) fwd_kernel(Args a) {
    constexpr int LH = D / 16;   // lanes per head: 16 values (8 pairs) each
    constexpr int HW = 32 / LH;  // heads per warp and step
    constexpr int STEP = HW * kUnroll;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ unsigned long long s_turn[D / 2];
    __shared__ __align__(16) float s_w[2][D], s_c[kWarps][D / 2], s_s[kWarps][D / 2];
    __shared__ __align__(8) unsigned long long s_bar[kWarps][FwdRing::kStages];
    __shared__ int s_abort;
    paged::after_previous();
    paged::let_next();
    load_turns(s_turn, a.freqs, a.rot / 2, threadIdx.x, 32 * kWarps);
    for (int i = threadIdx.x; i < 2 * D; i += 32 * kWarps)
        if (i < D || a.k.heads) s_w[i / D][i % D] = weight(i < D ? a.q.w : a.k.w, a.w32, i % D);
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w) FwdRing::init(s_bar[w]);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, item = lane % LH, hsub = lane / LH;
    const bool turns = item < a.rot / 16;  // the other items are not rotated
    int va, vb;
    vectors<D, INTERLEAVED>(item, a.rot / 2, va, vb);
    const int warp = threadIdx.x >> 5, Hq = a.q.heads, heads = Hq + a.k.heads;
    const unsigned units = (unsigned)a.tokens * a.splits, stride = gridDim.x * kWarps;
    auto token = [&](unsigned u) { return (int)(a.splits == 1 ? u : u / a.splits); };
    auto begin = [&](unsigned u) { return a.splits == 1 ? 0 : (int)(u % a.splits) * a.chunk; };
    // where a step that begins with head h of all ends: at that of q, of k, or of the unit
    auto length = [&](int h, int end) { return min(STEP, (h < Hq ? min(end, Hq) : end) - h); };
    ptx::Ctl ctl{&s_abort, a.status, kDefaultWaitLimit};
    FwdRing ring(s_bar[warp], ptx::saddr(s_ring) + warp * FwdRing::kBytes);
    unsigned u = blockIdx.x * kWarps + warp, nu = u;                    // the unit at hand, the one to be copied next
    int nh = begin(min(u, units - 1)), nhi = min(nh + a.chunk, heads);  // its heads that are left
    auto issue = [&] {
        if (nu >= units) return;
        const int t = token(nu), n = length(nh, nhi);
        const void *const src[1] = {nh < Hq ? a.q.x + t * a.q.xs + (size_t)nh * D : a.k.x + t * a.k.xs + (size_t)(nh - Hq) * D};
        ring.fill(lane, src, (uint32_t)n * D * 2);
        nh += n;
        if (nh >= nhi && (nu += stride) < units) {
            nh = begin(nu);
            nhi = min(nh + a.chunk, heads);
        }
    };
#pragma unroll 1
    for (int i = 0; i < FwdRing::kStages - 1; ++i) issue();
    int pos = u < units ? a.pos[token(u)] : 0;
    bool ok = true;
    for (; ok && u < units; u += stride) {
        const int t = token(u), h0 = begin(u), h1 = min(h0 + a.chunk, heads);
        warp_cos_sin(s_turn, a.rot / 2, lane, pos, a.mag, 1.f, s_c[warp], s_s[warp]);
        if (u + stride < units) pos = a.pos[token(u + stride)];
        float2 c[4], s[4];
        if (turns) {
            load_eight(s_c[warp] + item * 8, c);
            load_eight(s_s[warp] + item * 8, s);
        }
#pragma unroll 1
        for (int hb = h0, n; hb < h1; hb += n) {
            issue();
            const uint32_t stage = ring.wait(ctl);
            ok = stage != 0;
            if (!ok) break;
            n = length(hb, h1);
            const bool is_k = hb >= Hq;
            __nv_bfloat16 *dst = (is_k ? a.k.out + t * a.k.os + (size_t)(hb - Hq) * D : a.q.out + t * a.q.os + (size_t)hb * D);
            float2 wa[4], wb[4];
            load_eight(s_w[is_k] + va, wa);
            load_eight(s_w[is_k] + vb, wb);
            auto group = [&](int j) {
                const int i = j * HW + hsub;
                uint4 xa = make_uint4(0, 0, 0, 0), xb = xa;
                if (i < n) {
                    xa = ptx::ld_shared_v4(stage + i * D * 2 + 2 * va);
                    xb = ptx::ld_shared_v4(stage + i * D * 2 + 2 * vb);
                }
                float2 fa[4], fb[4];
                unpack(xa, fa);
                unpack(xb, fb);
                normalise<D>(fa, fb, wa, wb, a.eps);
                if (turns) turn_pairs<INTERLEAVED>(fa, fb, c, s);
                if (i < n) store_head<INTERLEAVED>(dst + (size_t)i * D, va, vb, a.wide, pack(fa), pack(fb));
            };
            if (n == STEP) {  // (whole: without a branch between them)
#pragma unroll
                for (int j = 0; j < kUnroll; ++j) group(j);
            } else {
#pragma unroll 1
                for (int j = 0; j * HW < n; ++j) group(j);
            }
            ring.release();
        }
    }
    ring.drain();
}

// The first q_ctas CTAs take q, the others k, so that a thread sums one weight's
// gradient (both cost it 16 more registers, and the second CTA of an SM).  A warp works
// through its units' steps, kBwdUnroll heads of every lane each, whose x and dy come by
// bulk copies two steps ahead.
template <int D>
using BwdRing = WarpRing<3, 2 * kBwdUnroll * 1024>;  // 32 lanes * 16 values, x and dy

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps, kBwdCtas) bwd_kernel(Args a) {
    constexpr int LH = D / 16, HW = 32 / LH, STEP = HW * kBwdUnroll;
    using R = BwdRing<D>;
    extern __shared__ __align__(128) uint8_t s_ring[];
    __shared__ unsigned long long s_turn[D / 2];
    __shared__ __align__(16) float s_w[D], s_c[kWarps][D / 2], s_s[kWarps][D / 2];
    __shared__ __align__(8) unsigned long long s_bar[kWarps][R::kStages];
    __shared__ int s_abort;
    const bool is_k = (int)blockIdx.x >= a.q_ctas;
    const Side x = is_k ? a.k : a.q;
    paged::after_previous();
    paged::let_next();
    load_turns(s_turn, a.freqs, a.rot / 2, threadIdx.x, 32 * kWarps);
    for (int i = threadIdx.x; i < D; i += 32 * kWarps) s_w[i] = weight(x.w, a.w32, i);
    if (threadIdx.x == 0) {
        for (int w = 0; w < kWarps; ++w) R::init(s_bar[w]);
        s_abort = 0;
        ptx::fence_mbar_init();
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = lane % LH, hsub = lane / LH;
    const bool turns = item < a.rot / 16;
    int va, vb;
    vectors<D, INTERLEAVED>(item, a.rot / 2, va, vb);
    float2 wa[4], wb[4], da[4], db[4];  // weights, and the sums of their gradients
    load_eight(s_w + va, wa);
    load_eight(s_w + vb, wb);
#pragma unroll
    for (int i = 0; i < 4; ++i) da[i] = db[i] = make_float2(0.f, 0.f);
    const int cta = is_k ? blockIdx.x - a.q_ctas : blockIdx.x, ctas = is_k ? gridDim.x - a.q_ctas : a.q_ctas;
    const unsigned units = (unsigned)a.tokens * x.splits, stride = ctas * kWarps;
    auto token = [&](unsigned u) { return (int)(x.splits == 1 ? u : u / x.splits); };
    auto begin = [&](unsigned u) { return x.splits == 1 ? 0 : (int)(u % x.splits) * x.chunk; };
    auto end = [&](int lo) { return min(lo + x.chunk, x.heads); };
    ptx::Ctl ctl{&s_abort, a.status, kDefaultWaitLimit};
    R ring(s_bar[warp], ptx::saddr(s_ring) + warp * R::kBytes);
    unsigned u = cta * kWarps + warp, nu = u;    // the unit at hand, and the one to be copied next
    int nh = begin(min(u, units - 1)), nhi = end(nh);  // its heads that are left
    auto issue = [&] {
        if (nu >= units) return;
        const int t = token(nu);
        const void *const src[2] = {x.x + t * x.xs + (size_t)nh * D, x.dy + t * x.ds + (size_t)nh * D};
        ring.fill(lane, src, (uint32_t)min(STEP, nhi - nh) * D * 2);
        nh += STEP;
        if (nh >= nhi && (nu += stride) < units) {
            nh = begin(nu);
            nhi = end(nh);
        }
    };
#pragma unroll 1
    for (int i = 0; i < R::kStages - 1; ++i) issue();
    int pos = u < units ? a.pos[token(u)] : 0;
    bool ok = true;
    for (; ok && u < units; u += stride) {
        const int t = token(u), lo = begin(u), hi = end(lo);
        warp_cos_sin(s_turn, a.rot / 2, lane, pos, a.mag, -1.f, s_c[warp], s_s[warp]);
        if (u + stride < units) pos = a.pos[token(u + stride)];
        float2 c[4], s[4];
        if (turns) {
            load_eight(s_c[warp] + item * 8, c);
            load_eight(s_s[warp] + item * 8, s);
        }
        __nv_bfloat16 *dst = x.out + t * x.os;
#pragma unroll 1
        for (int hb = lo; hb < hi; hb += STEP) {
            issue();
            const uint32_t stage = ring.wait(ctl);
            ok = stage != 0;
            if (!ok) break;
#pragma unroll
            for (int j = 0; j < kBwdUnroll; ++j) {
                if (hb + j * HW >= hi) break;  // (the warp alike)
                const int h = hb + j * HW + hsub;
                const uint32_t xs = stage + (j * HW + hsub) * D * 2, ys = xs + kBwdUnroll * 1024;
                uint4 v[4];
                v[0] = v[1] = v[2] = v[3] = make_uint4(0, 0, 0, 0);
                if (h < hi) {
                    v[0] = ptx::ld_shared_v4(xs + 2 * va);
                    v[1] = ptx::ld_shared_v4(xs + 2 * vb);
                    v[2] = ptx::ld_shared_v4(ys + 2 * va);
                    v[3] = ptx::ld_shared_v4(ys + 2 * vb);
                }
                float2 fa[4], fb[4], ga[4], gb[4], dot = make_float2(0.f, 0.f);
                unpack(v[0], fa);
                unpack(v[1], fb);
                unpack(v[2], ga);
                unpack(v[3], gb);
                const float2 r = both(inverse_rms<D>(fa, fb, a.eps));
                if (turns) turn_pairs<INTERLEAVED>(ga, gb, c, s);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    fa[i] = ptx::fmul2(fa[i], r);
                    fb[i] = ptx::fmul2(fb[i], r);
                    da[i] = ptx::ffma2(ga[i], fa[i], da[i]);
                    db[i] = ptx::ffma2(gb[i], fb[i], db[i]);
                    ga[i] = ptx::fmul2(ga[i], wa[i]);
                    gb[i] = ptx::fmul2(gb[i], wb[i]);
                    dot = ptx::ffma2(ga[i], fa[i], dot);
                    dot = ptx::ffma2(gb[i], fb[i], dot);
                }
                float sum = dot.x + dot.y;
#pragma unroll
                for (int o = 1; o < LH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float2 mean = both(sum * (-1.f / D));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ga[i] = ptx::fmul2(r, ptx::ffma2(fa[i], mean, ga[i]));
                    gb[i] = ptx::fmul2(r, ptx::ffma2(fb[i], mean, gb[i]));
                }
                if (h < hi) store_head<INTERLEAVED>(dst + (size_t)h * D, va, vb, a.wide, pack(ga), pack(gb));
            }
            ring.release();
        }
    }
    ring.drain();
    __syncthreads();  // (every warp has read its stages)
    float (*s_sum)[D] = reinterpret_cast<float (*)[D]>(s_ring);
    // the weight's gradient of this CTA, in an order fixed by the grid alone
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int o = LH; o < 32; o <<= 1) {
            da[i].x += __shfl_xor_sync(0xffffffffu, da[i].x, o);
            da[i].y += __shfl_xor_sync(0xffffffffu, da[i].y, o);
            db[i].x += __shfl_xor_sync(0xffffffffu, db[i].x, o);
            db[i].y += __shfl_xor_sync(0xffffffffu, db[i].y, o);
        }
        if (hsub == 0) {
            *reinterpret_cast<float2 *>(&s_sum[warp][va + 2 * i]) = da[i];
            *reinterpret_cast<float2 *>(&s_sum[warp][vb + 2 * i]) = db[i];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += 32 * kWarps) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += s_sum[w][i];
        a.part[(size_t)blockIdx.x * D + i] = sum;
    }
}

// The CTAs' sums of a weight's gradient: a warp 32 columns of every 32nd CTA, joined
// through shared memory by a warp for each column.  (fp32: 64-bit additions are slow
// enough here to show.  A thread of bwd_kernel adds tokens * heads / (its side's CTAs * 8 warps * the
// heads of a warp) terms in turn: some 30 at 32764 tokens of 32 heads of 128, 900 at a million, where the sum
// errs by 2^-14 of its terms' magnitudes at worst.)
constexpr int kSumWarps = 32;

__global__ void __launch_bounds__(32 * kSumWarps) weights_kernel(const float *part, int q_ctas, int ctas, int D,
                                                                 float *dwq, float *dwk) {
    __shared__ float s[kSumWarps][33];
    paged::after_previous();
    paged::let_next();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = blockIdx.x * 32;
    const int c0 = blockIdx.y ? q_ctas : 0, c1 = blockIdx.y ? ctas : q_ctas;
    float sum = 0.f;
    for (int c = c0 + warp; c < c1; c += 5 * kSumWarps) {
        float v[5];
#pragma unroll
        for (int j = 0; j < 5; ++j)
            v[j] = c + j * kSumWarps < c1 ? part[(size_t)(c + j * kSumWarps) * D + col + lane] : 0.f;
#pragma unroll
        for (int j = 0; j < 5; ++j) sum += v[j];
    }
    s[warp][lane] = sum;
    __syncthreads();
    sum = s[lane][warp];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) (blockIdx.y ? dwk : dwq)[col + warp] = sum;
}

// The gradient's CTAs, which leave a row of partial sums each: for q and k by what their
// tokens take where the GPU is full, one for every kWarps units where not.
int bwd_grid(Args *a, int D) {
    long long want[2], cost[2], cap = (long long)sm_count() * kBwdCtas;
    const long long steps = (long long)a->tokens * (a->q.heads + a->k.heads) * D / (512 * kBwdUnroll);
    if (steps >= kBwdWaves * kBwdWaveSteps * kWarps * cap) cap *= kBwdWaves;
    const int HW = 32 / (D / 16);
    Side *sides[2] = {&a->q, &a->k};
    for (int i = 0; i < 2; ++i) {
        Side &s = *sides[i];
        want[i] = cost[i] = 0;
        if (s.heads == 0) continue;
        // of a token: steps, and the heads of every lane
        cost[i] = (s.heads + HW * kBwdUnroll - 1) / (HW * kBwdUnroll) + (s.heads + HW - 1) / HW;
        split_heads(s.heads, a->tokens, D, kBwdUnroll, &s.chunk, &s.splits);
        want[i] = ((long long)a->tokens * s.splits + kWarps - 1) / kWarps;
    }
    if (want[0] + want[1] > cap) {
        long long nk = cap * cost[1] / (cost[0] + cost[1]);
        if (a->k.heads && nk < 1) nk = 1;
        if (nk > want[1]) nk = want[1];
        want[1] = nk;
        if (want[0] > cap - nk) want[0] = cap - nk;
    }
    a->q_ctas = (int)want[0];
    return (int)(want[0] + want[1]);
}

int check(const Args &a, int D, int interleaved, int weight_bits) {
    if (!a.pos || !a.freqs || a.tokens < 1 || a.q.heads < 1 || a.k.heads < 0) return MOBA_ERR_INVALID_ARG;
    if (!a.q.w || (a.k.heads && !a.k.w)) return MOBA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return MOBA_ERR_UNSUPPORTED;
    if (a.rot < 16 || a.rot > D || a.rot % 16 != 0) return MOBA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return MOBA_ERR_INVALID_ARG;
    if (weight_bits != 16 && weight_bits != 32) return MOBA_ERR_INVALID_ARG;
    if (!std::isfinite(a.mag) || !(a.eps >= 1e-12f) || !std::isfinite(a.eps)) return MOBA_ERR_INVALID_ARG;
    if (a.q.heads > 65535 || a.k.heads > 65535) return MOBA_ERR_UNSUPPORTED;
    if (reinterpret_cast<uintptr_t>(a.pos) & 3 || reinterpret_cast<uintptr_t>(a.freqs) & 7)
        return MOBA_ERR_INVALID_ARG;
    const uintptr_t w = reinterpret_cast<uintptr_t>(a.q.w) | (a.k.heads ? reinterpret_cast<uintptr_t>(a.k.w) : 0);
    if (w & (weight_bits / 8 - 1)) return MOBA_ERR_INVALID_ARG;
    return MOBA_OK;
}

// whether every head of the results is aligned to 32 bytes
bool wide(const Args &a) {
    uintptr_t w = 0;
    for (const Side *s : {&a.q, &a.k})
        if (s->heads) w |= reinterpret_cast<uintptr_t>(s->out) | (uintptr_t)(2 * s->os);
    return (w & 31) == 0;
}

struct Area {
    const void *p;
    long long stride, width;  // bytes
};
Area area(const void *p, long long stride, int heads, int D) { return {p, 2 * stride, 2ll * heads * D}; }

// an output against what else the call reads and writes; `own`: its own operand, which it may be
// in place (that goes by the operand, not by its address: another one may have the same)
bool collides(const Area &out, const Area &in, bool own, long long tokens) {
    if (!in.p || !out.p) return false;
    if (own && out.p == in.p && out.stride == in.stride) return false;
    return overlaps(out.p, out.stride, out.width, in.p, in.stride, in.width, tokens);
}

// `bytes` at p in one piece, and whether an area's rows meet them, or another piece does
struct Piece {
    const void *p;
    long long bytes;
};
bool collides(const Area &rows, const Piece &x, long long tokens) {
    if (!rows.p || !x.p) return false;
    const intptr_t r = reinterpret_cast<intptr_t>(rows.p), lo = reinterpret_cast<intptr_t>(x.p), hi = lo + x.bytes;
    const long long first = lo < r + rows.width ? 0 : (lo - r - rows.width) / rows.stride + 1;  // row that ends behind lo
    return first < tokens && r + first * rows.stride < hi;
}
bool collides(const Piece &x, const Piece &y) {
    const intptr_t a = reinterpret_cast<intptr_t>(x.p), b = reinterpret_cast<intptr_t>(y.p);
    return x.p && y.p && a < b + y.bytes && b < a + x.bytes;
}

// What a call reads beside q, k and their gradients.
struct Small {
    Piece all[4];
    Small(const Args &a, int D)
        : all{{a.q.w, (a.w32 ? 4ll : 2ll) * D}, {a.k.heads ? a.k.w : nullptr, (a.w32 ? 4ll : 2ll) * D}, {a.pos, 4ll * a.tokens},
              {a.freqs, 4ll * a.rot}} {}
    bool meet(const Area &out, long long tokens) const {
        for (const Piece &x : all)
            if (collides(out, x, tokens)) return true;
        return false;
    }
};

template <int D>
cudaError_t launch_fwd(const Args &a, bool interleaved, cudaStream_t st) {
    const long long units = (long long)a.tokens * a.splits;
    const long long want = (units + kWarps - 1) / kWarps, once = (long long)sm_count() * kFwdCtas;
    const long long steps = (long long)a.tokens * (a.q.heads + a.k.heads) * D / (512 * kUnroll);
    const long long waves = std::min(std::max(steps / (kWaveSteps * kWarps * once), 1ll), (long long)kFwdWaves), cap = waves * once;
    const int grid = (int)(want < cap ? want : cap);
    constexpr int bytes = kWarps * FwdRing::kBytes;
    const cudaError_t rc = interleaved ? paged::allow_smem<fwd_kernel<D, true>>(bytes) : paged::allow_smem<fwd_kernel<D, false>>(bytes);
    if (rc != cudaSuccess) return rc;
    note_launches(1);
    return interleaved ? paged::launch_after(fwd_kernel<D, true>, dim3(grid), dim3(32 * kWarps), bytes, st, a)
                       : paged::launch_after(fwd_kernel<D, false>, dim3(grid), dim3(32 * kWarps), bytes, st, a);
}

template <int D>
cudaError_t launch_bwd(const Args &a, int grid, bool interleaved, float *dwq, float *dwk, cudaStream_t st) {
    constexpr int bytes = kWarps * BwdRing<D>::kBytes;
    cudaError_t rc = interleaved ? paged::allow_smem<bwd_kernel<D, true>>(bytes) : paged::allow_smem<bwd_kernel<D, false>>(bytes);
    if (rc != cudaSuccess) return rc;
    note_launches(2);
    rc = interleaved ? paged::launch_after(bwd_kernel<D, true>, dim3(grid), dim3(32 * kWarps), bytes, st, a)
                     : paged::launch_after(bwd_kernel<D, false>, dim3(grid), dim3(32 * kWarps), bytes, st, a);
    if (rc != cudaSuccess) return rc;
    return paged::launch_after(weights_kernel, dim3(D / 32, dwk ? 2 : 1), dim3(32 * kSumWarps), 0, st,
                               (const float *)a.part, a.q_ctas, grid, D, dwq, dwk);
}

}  // namespace qk_norm
}  // namespace moba

using namespace moba;
using namespace moba::qk_norm;

MOBA_EXPORT int moba_qk_norm_rope(const void *q, const void *k, void *q_out, void *k_out, const void *q_weight,
                                  const void *k_weight, int weight_bits, float eps, const int32_t *positions,
                                  const double *freqs, int tokens, int Hq, int Hk, int D, int rot_dim,
                                  int interleaved, float magnitude, long long q_stride, long long k_stride,
                                  long long q_out_stride, long long k_out_stride, void *stream) {
    Args a = {};
    a.q = {static_cast<const __nv_bfloat16 *>(q), nullptr, static_cast<__nv_bfloat16 *>(q_out), q_weight, q_stride, 0,
           q_out_stride, Hq};
    a.k = {static_cast<const __nv_bfloat16 *>(k), nullptr, static_cast<__nv_bfloat16 *>(k_out), k_weight, k_stride, 0,
           k_out_stride, Hk};
    a.pos = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.rot = rot_dim;
    a.w32 = weight_bits == 32;
    a.eps = eps;
    a.mag = magnitude;
    int rc = check(a, D, interleaved, weight_bits);
    for (Side *s : {&a.q, &a.k}) {
        if (s == &a.k && Hk == 0) break;
        if (rc == MOBA_OK) rc = check_rows(s->x, s->heads, D, tokens, &s->xs);
        if (rc == MOBA_OK) rc = check_rows(s->out, s->heads, D, tokens, &s->os);
    }
    if (rc != MOBA_OK) return rc;
    const Area qi = area(q, a.q.xs, Hq, D), qo = area(q_out, a.q.os, Hq, D);
    const Area ki = Hk ? area(k, a.k.xs, Hk, D) : Area{}, ko = Hk ? area(k_out, a.k.os, Hk, D) : Area{};
    const Small small(a, D);
    if (collides(qo, qi, true, tokens) || collides(qo, ki, false, tokens) || collides(ko, qi, false, tokens) ||
        collides(ko, ki, true, tokens) || collides(ko, qo, false, tokens) || small.meet(qo, tokens) || small.meet(ko, tokens))
        return MOBA_ERR_INVALID_ARG;
    a.wide = wide(a);
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    split_heads(Hq + Hk, tokens, D, kUnroll, &a.chunk, &a.splits);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_result(D == 64 ? launch_fwd<64>(a, interleaved != 0, st) : launch_fwd<128>(a, interleaved != 0, st));
}

MOBA_EXPORT size_t moba_qk_norm_rope_bwd_workspace_size(int tokens, int Hq, int Hk, int D) {
    if (tokens < 1 || Hq < 1 || Hk < 0 || (D != 64 && D != 128) || Hq > 65535 || Hk > 65535) return 0;
    Args a = {};
    a.tokens = tokens;
    a.q.heads = Hq;
    a.k.heads = Hk;
    return sizeof(float) * D * (size_t)bwd_grid(&a, D);
}

MOBA_EXPORT int moba_qk_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *q, const void *k,
                                      const void *q_weight, const void *k_weight, void *dq, void *dk,
                                      float *dq_weight, float *dk_weight, int weight_bits, float eps,
                                      const int32_t *positions, const double *freqs, int tokens, int Hq, int Hk,
                                      int D, int rot_dim, int interleaved, float magnitude, long long dq_out_stride,
                                      long long dk_out_stride, long long q_stride, long long k_stride,
                                      long long dq_stride, long long dk_stride, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    Args a = {};
    a.q = {static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(dq_out),
           static_cast<__nv_bfloat16 *>(dq), q_weight, q_stride, dq_out_stride, dq_stride, Hq};
    a.k = {static_cast<const __nv_bfloat16 *>(k), static_cast<const __nv_bfloat16 *>(dk_out),
           static_cast<__nv_bfloat16 *>(dk), k_weight, k_stride, dk_out_stride, dk_stride, Hk};
    a.pos = positions;
    a.freqs = freqs;
    a.tokens = tokens;
    a.rot = rot_dim;
    a.w32 = weight_bits == 32;
    a.eps = eps;
    a.mag = magnitude;
    int rc = check(a, D, interleaved, weight_bits);
    for (Side *s : {&a.q, &a.k}) {
        if (s == &a.k && Hk == 0) break;
        if (rc == MOBA_OK) rc = check_rows(s->x, s->heads, D, tokens, &s->xs);
        if (rc == MOBA_OK) rc = check_rows(s->dy, s->heads, D, tokens, &s->ds);
        if (rc == MOBA_OK) rc = check_rows(s->out, s->heads, D, tokens, &s->os);
    }
    if (rc != MOBA_OK) return rc;
    if (!dq_weight || (Hk && !dk_weight) ||
        ((reinterpret_cast<uintptr_t>(dq_weight) | (Hk ? reinterpret_cast<uintptr_t>(dk_weight) : 0)) & 3))
        return MOBA_ERR_INVALID_ARG;
    const Area qx = area(q, a.q.xs, Hq, D), qy = area(dq_out, a.q.ds, Hq, D), qo = area(dq, a.q.os, Hq, D);
    const Area kx = Hk ? area(k, a.k.xs, Hk, D) : Area{}, ky = Hk ? area(dk_out, a.k.ds, Hk, D) : Area{};
    const Area ko = Hk ? area(dk, a.k.os, Hk, D) : Area{};
    if (collides(qo, qy, true, tokens) || collides(qo, ky, false, tokens) || collides(ko, ky, true, tokens) ||
        collides(ko, qy, false, tokens) || collides(ko, qo, false, tokens))
        return MOBA_ERR_INVALID_ARG;
    const Piece wq = {dq_weight, 4ll * D}, wk = {Hk ? dk_weight : nullptr, 4ll * D};
    for (const Area &in : {qx, kx})
        if (collides(qo, in, false, tokens) || collides(ko, in, false, tokens)) return MOBA_ERR_INVALID_ARG;
    for (const Area &rows : {qx, kx, qy, ky, qo, ko})
        if (collides(rows, wq, tokens) || collides(rows, wk, tokens)) return MOBA_ERR_INVALID_ARG;
    const Small small(a, D);
    for (const Piece &x : small.all)
        if (collides(x, wq) || collides(x, wk)) return MOBA_ERR_INVALID_ARG;
    if (collides(wq, wk) || small.meet(qo, tokens) || small.meet(ko, tokens)) return MOBA_ERR_INVALID_ARG;
    a.wide = wide(a);
    const int grid = bwd_grid(&a, D);
    const size_t need = sizeof(float) * D * (size_t)grid;
    if (workspace && (workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return MOBA_ERR_WORKSPACE;
    a.status = status_word();
    if (!a.status) return cuda_result(cudaErrorInvalidDevice);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    void *own = nullptr;
    if (!workspace) {
        const cudaError_t e = cudaMallocAsync(&own, need, st);
        if (e != cudaSuccess) return cuda_result(e);
        workspace = own;
    }
    a.part = static_cast<float *>(workspace);
    cudaError_t e = D == 64 ? launch_bwd<64>(a, grid, interleaved != 0, dq_weight, Hk ? dk_weight : nullptr, st)
                            : launch_bwd<128>(a, grid, interleaved != 0, dq_weight, Hk ? dk_weight : nullptr, st);
    if (own) {
        const cudaError_t f = cudaFreeAsync(own, st);
        if (e == cudaSuccess) e = f;
    }
    return cuda_result(e);
}
