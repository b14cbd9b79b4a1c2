// moba_rope.cu -- rotary positions of q and k, and the gradient of the rotation.
//
// Pages: "When a MoBA reproduction will not run" (mhpq.cn/news/582794) section
// 3.3 asks where positions enter MoBA; here they enter before the gate, by
// rotating q and k, so that the pooled keys are means of rotated keys.
//
// A pair (a, b) of a head turns by angle pos * freq[pair]:
//   a' = m (a cos - b sin),  b' = m (b cos + a sin);  the gradient is the
// transpose, the same with -sin.  The phase is held in turns as a 64-bit
// fixed-point fraction: frac(freq / 2 pi) * 2^64 times the position, modulo
// 2^64, is the position's phase exactly up to pos * 2^-56 turns (the rounding
// of freq / 2 pi in 64 bits), so far positions lose nothing to range
// reduction.  cos and sin are then fp32 of a phase in [-1/2, 1/2] turns.
//
// Bound: HBM (two bytes read and two written per value).  A warp takes one
// token and a run of its heads; a lane keeps the cos and sin of its eight
// pairs in registers for all of them, so the phases cost little.  Measured: 165 us
// for 32768 tokens of 64 heads of 128, 6.5 TB/s, 0.97 of the copy rate; 85 us, 0.93,
// for the gradient of 32764 tokens of 32 heads, half of each rotated.  A decode step's
// tokens are bound by latency and the call: 1, 64, 256 tokens of 40 heads 2.9, 3.4, 3.3 us
// in a graph, 10.6 by a call from Python.
#include <cmath>

#include "moba.h"
#include "moba_rope.cuh"

namespace moba {
namespace rope {

constexpr int kWarps = 8;
constexpr int kUnroll = 4;  // heads whose loads a lane has in flight

struct Args {
    const __nv_bfloat16 *q, *k;
    __nv_bfloat16 *qo, *ko;
    const int32_t *pos;
    const double *freqs;
    long long q_stride, k_stride, qo_stride, ko_stride;  // elements between tokens
    int tokens, Hq, Hk, rot;
    int chunk, splits;  // heads per unit, units per token
    float mag, sin_sign;
};

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(32 * kWarps) rope_kernel(Args a) {
    constexpr int LH = D / 16;   // lanes per head: 16 values (8 pairs) each
    constexpr int HW = 32 / LH;  // heads per warp and step
    __shared__ unsigned long long s_turn[D / 2];
    const int half = a.rot / 2;
    load_turns(s_turn, a.freqs, half, threadIdx.x, 32 * kWarps);
    __syncthreads();
    const int lane = threadIdx.x & 31, item = lane % LH, hsub = lane / LH;
    const bool turns = item < a.rot / 16;  // the other items copy the unrotated rest
    int va, vb;  // where the item's two 16-byte vectors start inside the head
    vectors<D, INTERLEAVED>(item, half, va, vb);
    const long long units = (long long)a.tokens * a.splits;
    for (long long u = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units;
         u += (long long)gridDim.x * kWarps) {
        const int t = (int)(u / a.splits);
        const int h0 = (int)(u % a.splits) * a.chunk, h1 = min(h0 + a.chunk, a.Hq + a.Hk);
        float c[8], s[8];
        if (turns) cos_sin(s_turn + item * 8, __ldg(a.pos + t), a.mag, a.sin_sign, c, s);
        for (int hb = h0; hb < h1; hb += HW * kUnroll) {
            uint4 xa[kUnroll], xb[kUnroll];
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int h = hb + j * HW + hsub;
                if (h < h1) {
                    const __nv_bfloat16 *src = h < a.Hq ? a.q + t * a.q_stride + (size_t)h * D
                                                        : a.k + t * a.k_stride + (size_t)(h - a.Hq) * D;
                    xa[j] = *reinterpret_cast<const uint4 *>(src + va);
                    xb[j] = *reinterpret_cast<const uint4 *>(src + vb);
                }
            }
#pragma unroll
            for (int j = 0; j < kUnroll; ++j) {
                const int h = hb + j * HW + hsub;
                if (h >= h1) continue;
                if (turns) {
                    __nv_bfloat162 *pa = reinterpret_cast<__nv_bfloat162 *>(&xa[j]);
                    __nv_bfloat162 *pb = reinterpret_cast<__nv_bfloat162 *>(&xb[j]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 fa = __bfloat1622float2(pa[e]), fb = __bfloat1622float2(pb[e]);
                        if (INTERLEAVED) {  // pairs inside each vector
                            pa[e] = __floats2bfloat162_rn(fmaf(fa.x, c[e], -fa.y * s[e]),
                                                          fmaf(fa.y, c[e], fa.x * s[e]));
                            pb[e] = __floats2bfloat162_rn(fmaf(fb.x, c[4 + e], -fb.y * s[4 + e]),
                                                          fmaf(fb.y, c[4 + e], fb.x * s[4 + e]));
                        } else {  // pair i: value i of the first vector, value i of the second
                            pa[e] = __floats2bfloat162_rn(fmaf(fa.x, c[2 * e], -fb.x * s[2 * e]),
                                                          fmaf(fa.y, c[2 * e + 1], -fb.y * s[2 * e + 1]));
                            pb[e] = __floats2bfloat162_rn(fmaf(fb.x, c[2 * e], fa.x * s[2 * e]),
                                                          fmaf(fb.y, c[2 * e + 1], fa.y * s[2 * e + 1]));
                        }
                    }
                }
                __nv_bfloat16 *dst = h < a.Hq ? a.qo + t * a.qo_stride + (size_t)h * D
                                              : a.ko + t * a.ko_stride + (size_t)(h - a.Hq) * D;
                *reinterpret_cast<uint4 *>(dst + va) = xa[j];
                *reinterpret_cast<uint4 *>(dst + vb) = xb[j];
            }
        }
    }
}

template <int D>
static cudaError_t launch(const Args &a, bool interleaved, cudaStream_t st) {
    const long long units = (long long)a.tokens * a.splits;
    const long long want = (units + kWarps - 1) / kWarps;
    const long long cap = (long long)sm_count() * 8;
    const int grid = (int)(want < cap ? want : cap);
    if (interleaved) rope_kernel<D, true><<<grid, 32 * kWarps, 0, st>>>(a);
    else rope_kernel<D, false><<<grid, 32 * kWarps, 0, st>>>(a);
    note_launches(1);
    return cudaGetLastError();
}

static int run(const void *q, const void *k, void *qo, void *ko, const int32_t *pos,
               const double *freqs, int tokens, int Hq, int Hk, int D, int rot, int interleaved,
               float mag, long long qs, long long ks, long long qos, long long kos, float sign,
               void *stream) {
    if (!q || !qo || !pos || !freqs || tokens < 1 || Hq < 1 || Hk < 0) return MOBA_ERR_INVALID_ARG;
    if (Hk > 0 && (!k || !ko)) return MOBA_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return MOBA_ERR_UNSUPPORTED;
    if (rot < 16 || rot > D || rot % 16 != 0) return MOBA_ERR_INVALID_ARG;
    if (interleaved != 0 && interleaved != 1) return MOBA_ERR_INVALID_ARG;
    if (!std::isfinite(mag)) return MOBA_ERR_INVALID_ARG;
    if (Hq > 65535 || Hk > 65535) return MOBA_ERR_UNSUPPORTED;
    if (misaligned16(q) || misaligned16(qo) || (Hk && (misaligned16(k) || misaligned16(ko))))
        return MOBA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(pos) & 3) || (reinterpret_cast<uintptr_t>(freqs) & 7))
        return MOBA_ERR_INVALID_ARG;
    const long long wq = (long long)Hq * D, wk = (long long)Hk * D;
    if (qs == 0) qs = wq;
    if (qos == 0) qos = wq;
    if (ks == 0) ks = wk;
    if (kos == 0) kos = wk;
    if (qs < wq || qos < wq || qs % 8 || qos % 8) return MOBA_ERR_INVALID_ARG;
    if (Hk && (ks < wk || kos < wk || ks % 8 || kos % 8)) return MOBA_ERR_INVALID_ARG;
    const long long lim = 1ll << 40;
    if (qs > lim / tokens || qos > lim / tokens || ks > lim / tokens || kos > lim / tokens)
        return MOBA_ERR_UNSUPPORTED;
    // an output may be its own input (in place), and overlaps nothing else
    if ((q != qo || qs != qos) && overlaps(q, 2 * qs, 2 * wq, qo, 2 * qos, 2 * wq, tokens))
        return MOBA_ERR_INVALID_ARG;
    if (Hk) {
        if ((k != ko || ks != kos) && overlaps(k, 2 * ks, 2 * wk, ko, 2 * kos, 2 * wk, tokens))
            return MOBA_ERR_INVALID_ARG;
        if (overlaps(q, 2 * qs, 2 * wq, ko, 2 * kos, 2 * wk, tokens) ||
            overlaps(qo, 2 * qos, 2 * wq, k, 2 * ks, 2 * wk, tokens) ||
            overlaps(qo, 2 * qos, 2 * wq, ko, 2 * kos, 2 * wk, tokens))
            return MOBA_ERR_INVALID_ARG;
    }
    Args a;
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.k = static_cast<const __nv_bfloat16 *>(k);
    a.qo = static_cast<__nv_bfloat16 *>(qo);
    a.ko = static_cast<__nv_bfloat16 *>(ko);
    a.pos = pos;
    a.freqs = freqs;
    a.q_stride = qs;
    a.k_stride = ks;
    a.qo_stride = qos;
    a.ko_stride = kos;
    a.tokens = tokens;
    a.Hq = Hq;
    a.Hk = Hk;
    a.rot = rot;
    a.mag = mag;
    a.sin_sign = sign;
    // a token's heads in one warp when there are tokens enough to fill the GPU
    // (the phases are computed once), else spread over warps, a step of loads each
    const int heads = Hq + Hk, step = (32 / (D / 16)) * kUnroll;
    const int most = (heads + step - 1) / step;
    const long long fill = (long long)sm_count() * 16;
    long long splits = (fill + tokens - 1) / tokens;
    if (splits > most) splits = most;
    const int per = ((int)((most + splits - 1) / splits)) * step;
    a.chunk = per;
    a.splits = (heads + per - 1) / per;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_result(D == 64 ? launch<64>(a, interleaved != 0, st)
                               : launch<128>(a, interleaved != 0, st));
}

}  // namespace rope
}  // namespace moba

MOBA_EXPORT int moba_rope(const void *q, const void *k, void *q_out, void *k_out,
                          const int32_t *positions, const double *freqs, int tokens, int Hq, int Hk,
                          int D, int rot_dim, int interleaved, float magnitude, long long q_stride,
                          long long k_stride, long long q_out_stride, long long k_out_stride,
                          void *stream) {
    return moba::rope::run(q, k, q_out, k_out, positions, freqs, tokens, Hq, Hk, D, rot_dim,
                           interleaved, magnitude, q_stride, k_stride, q_out_stride, k_out_stride,
                           1.f, stream);
}

MOBA_EXPORT int moba_rope_bwd(const void *dq_out, const void *dk_out, void *dq, void *dk,
                              const int32_t *positions, const double *freqs, int tokens, int Hq,
                              int Hk, int D, int rot_dim, int interleaved, float magnitude,
                              long long dq_out_stride, long long dk_out_stride, long long dq_stride,
                              long long dk_stride, void *stream) {
    return moba::rope::run(dq_out, dk_out, dq, dk, positions, freqs, tokens, Hq, Hk, D, rot_dim,
                           interleaved, magnitude, dq_out_stride, dk_out_stride, dq_stride,
                           dk_stride, -1.f, stream);
}

MOBA_EXPORT int moba_rope_frequencies(double *freqs, int rot_dim, double base, int scaling,
                                      double factor, double original_length, double slow_turns,
                                      double fast_turns) {
    if (!freqs || rot_dim < 2 || rot_dim % 2 || !(base > 1.0) || !std::isfinite(base))
        return MOBA_ERR_INVALID_ARG;
    if (scaling < MOBA_ROPE_PLAIN || scaling > MOBA_ROPE_BANDS) return MOBA_ERR_INVALID_ARG;
    if (scaling != MOBA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return MOBA_ERR_INVALID_ARG;
    if (scaling == MOBA_ROPE_BASE && rot_dim <= 2) return MOBA_ERR_INVALID_ARG;
    if (scaling == MOBA_ROPE_BANDS &&
        (!(original_length > 0.0) || !std::isfinite(original_length) || !(slow_turns >= 0.0) ||
         !(fast_turns > slow_turns) || !std::isfinite(fast_turns)))
        return MOBA_ERR_INVALID_ARG;
    const double pi = 3.14159265358979323846;
    if (scaling == MOBA_ROPE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == MOBA_ROPE_LINEAR) f /= factor;
        if (scaling == MOBA_ROPE_BANDS) {
            const double turns = original_length * f / (2 * pi);
            double keep = (turns - slow_turns) / (fast_turns - slow_turns);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            f = f * keep + f / factor * (1 - keep);
        }
        freqs[i] = f;
    }
    return MOBA_OK;
}
