// moba_rope.cuh -- what the kernels that rotate heads to their positions share: the
// layout of a head over lanes, the phases, and the host checks of their operands.
#pragma once

#include <math_constants.h>

#include "moba_internal.cuh"

namespace moba {
namespace rope {

// A head of D values lies on D / 16 lanes, 16 values each, in two 16-byte vectors:
// eight pairs where the lane's values are rotated (its item is below rot / 16), else
// 16 neighbours of the rest.
template <int D, bool INTERLEAVED>
__device__ __forceinline__ void vectors(int item, int half, int &va, int &vb) {
    if (item >= half / 8 || INTERLEAVED) {
        va = item * 16;
        vb = va + 8;
    } else {
        va = item * 8;
        vb = va + half;
    }
}

// frac(freq / 2 pi) * 2^64 of every pair: turns per position in fixed point
__device__ __forceinline__ void load_turns(unsigned long long *turn, const double *freqs, int half,
                                           int thread, int threads) {
    for (int i = thread; i < half; i += threads) {
        const double t = __ldg(freqs + i) * 0.15915494309189533577;  // turns per position
        turn[i] = __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
    }
}

// mag * cos and mag * sign * sin of position p, of the eight pairs at turn
__device__ __forceinline__ void cos_sin(const unsigned long long *turn, long long p, float mag,
                                        float sign, float (&c)[8], float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const unsigned long long phase = turn[i] * (unsigned long long)p;
        // the upper 32 bits as a signed fraction of half a turn
        const float x = (float)(int)(phase >> 32) * 4.656612873077392578125e-10f;
        sincospif(x, &s[i], &c[i]);
        s[i] *= mag * sign;
        c[i] *= mag;
    }
}

// The lane's two vectors in 32 bits, a its first eight values, b its last eight.
__device__ __forceinline__ void unpack(const uint4 &v, float (&f)[8]) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = __bfloat1622float2(p[e]);
        f[2 * e] = x.x;
        f[2 * e + 1] = x.y;
    }
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint4 v;
    __nv_bfloat162 *p = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    return v;
}

// The eight pairs turned: pair i is (a[i], b[i]), or neighbours of a and then of b.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(float (&a)[8], float (&b)[8], const float (&c)[8],
                                           const float (&s)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &x = INTERLEAVED ? (i < 4 ? a[2 * i] : b[2 * i - 8]) : a[i];
        float &y = INTERLEAVED ? (i < 4 ? a[2 * i + 1] : b[2 * i - 7]) : b[i];
        const float u = fmaf(x, c[i], -y * s[i]), v = fmaf(y, c[i], x * s[i]);
        x = u;
        y = v;
    }
}

// 1 / sqrt(mean x^2 + eps) of the head whose values are on `lanes` neighbouring
// lanes.  All lanes of the warp call it.
template <int D>
__device__ __forceinline__ float inverse_rms(const float (&a)[8], const float (&b)[8], float eps) {
    constexpr int LH = D / 16;
    auto squares = [&](float f) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = a[i] * f, y = b[i] * f;
            ss = fmaf(x, x, ss);
            ss = fmaf(y, y, ss);
        }
#pragma unroll
        for (int o = 1; o < LH; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        return ss;
    };
    const float ss = squares(1.f);
    float r = rsqrtf(fmaf(ss, 1.f / D, eps));
    const bool big = !(ss < CUDART_INF_F);
    if (__any_sync(0xffffffffu, big)) {
        // squares out of fp32's range: of values times 2^-70 (eps is nothing beside them)
        const float t = squares(0x1p-70f);
        if (big) r = rsqrtf(t * (1.f / D)) * 0x1p-70f;
    }
    return r;
}

__device__ __forceinline__ float weight(const void *w, int w32, int d) {
    return w32 ? __ldg(static_cast<const float *>(w) + d)
               : __bfloat162float(__ldg(static_cast<const __nv_bfloat16 *>(w) + d));
}

// the lane's 16 weights
__device__ __forceinline__ void load_weights(const float *w, int va, int vb, float (&wa)[8], float (&wb)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4 *>(wa + i) = *reinterpret_cast<const float4 *>(w + va + i);
        *reinterpret_cast<float4 *>(wb + i) = *reinterpret_cast<const float4 *>(w + vb + i);
    }
}

// a head over its root mean square, times the weights
template <int D>
__device__ __forceinline__ void normalise(float (&a)[8], float (&b)[8], const float (&wa)[8], const float (&wb)[8],
                                          float eps) {
    const float r = inverse_rms<D>(a, b, eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = a[i] * r * wa[i];
        b[i] = b[i] * r * wb[i];
    }
}

// Units of a call: all heads of a token in one warp when there are tokens enough to
// fill the GPU (the phases are computed once), else spread over warps, a step of loads
// (`unroll` heads of every lane) each.
inline void split_heads(int heads, int tokens, int D, int unroll, int *chunk, int *splits) {
    const int step = (32 / (D / 16)) * unroll, most = (heads + step - 1) / step;
    long long n = ((long long)sm_count() * 16 + tokens - 1) / tokens;
    if (n > most) n = most;
    *chunk = ((int)((most + n - 1) / n)) * step;
    *splits = (heads + *chunk - 1) / *chunk;
}

// Whether two areas of `rows` rows overlap in memory: wx bytes every sx bytes
// from x, wy bytes every sy from y.
inline bool overlaps(const void *x, long long sx, long long wx, const void *y, long long sy,
                     long long wy, long long rows) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    const uintptr_t a1 = a + (uintptr_t)((rows - 1) * sx + wx);
    const uintptr_t b1 = b + (uintptr_t)((rows - 1) * sy + wy);
    if (a1 <= b || b1 <= a) return false;
    if (sx != sy) return true;
    // equal strides: rows may lie between one another (slices of one projection)
    const uintptr_t s = (uintptr_t)sx, d = b >= a ? (b - a) % s : (s - (a - b) % s) % s;
    return d < (uintptr_t)wx || s - d < (uintptr_t)wy;
}

// Tokens of `heads` heads of D values, *stride elements apart (0: dense): MOBA_OK, or
// why not.
inline int check_rows(const void *p, int heads, int D, int tokens, long long *stride) {
    if (!p || misaligned16(p)) return MOBA_ERR_INVALID_ARG;
    const long long w = (long long)heads * D;
    if (*stride == 0) *stride = w;
    if (*stride < w || *stride % 8) return MOBA_ERR_INVALID_ARG;
    return *stride > (1ll << 40) / tokens ? MOBA_ERR_UNSUPPORTED : MOBA_OK;
}

}  // namespace rope
}  // namespace moba
