// moba_rope.cuh -- what the kernels that rotate heads to their positions share: the
// layout of a head over lanes, the phases, and the host checks of their operands.
#pragma once

#include <math_constants.h>

#include "moba_internal.cuh"
#include "moba_ptx.cuh"

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
// (Plain loads here and in weight(): see launch_after.)
__device__ __forceinline__ void load_turns(unsigned long long *turn, const double *freqs, int half,
                                           int thread, int threads) {
    for (int i = thread; i < half; i += threads) {
        const double t = freqs[i] * 0.15915494309189533577;  // turns per position
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

// The lane's two vectors of a head to memory; neighbours (the pairs interleaved) as one of
// 32 bytes, a whole sector, where every head is aligned to that (wide).
template <bool INTERLEAVED>
__device__ __forceinline__ void store_head(__nv_bfloat16 *p, int va, int vb, bool wide, const uint4 &a, const uint4 &b) {
    if (INTERLEAVED && wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + va), "r"(a.x), "r"(a.y),
                     "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        *reinterpret_cast<uint4 *>(p + va) = a;
        *reinterpret_cast<uint4 *>(p + vb) = b;
    }
}

// The lane's two vectors in 32 bits, a its first eight values, b its last eight, two to a
// packed operation.
__device__ __forceinline__ void unpack(const uint4 &v, float2 (&f)[4]) {
    const __nv_bfloat162 *p = reinterpret_cast<const __nv_bfloat162 *>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __bfloat1622float2(p[e]);
}
__device__ __forceinline__ uint4 pack(const float2 (&f)[4]) {
    uint4 v;
    __nv_bfloat162 *p = reinterpret_cast<__nv_bfloat162 *>(&v);
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = __floats2bfloat162_rn(f[e].x, f[e].y);
    return v;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 minus(float2 x) { return make_float2(-x.x, -x.y); }

// mag * cos and mag * sign * sin of position p for all pairs, by the warp's lanes, left in
// c and s (of the warp alone); then the lane's eight from there.  (A lane's own pairs are
// those of every head of the warp: made lane by lane they cost four to eight times as much.)
__device__ __forceinline__ void warp_cos_sin(const unsigned long long *turn, int half, int lane, long long p,
                                             float mag, float sign, float *c, float *s) {
    __syncwarp();  // (the token before has been read)
    for (int i = lane; i < half; i += 32) {
        const unsigned long long phase = turn[i] * (unsigned long long)p;
        // the upper 32 bits as a signed fraction of half a turn
        const float x = (float)(int)(phase >> 32) * 4.656612873077392578125e-10f;
        float sn, cs;
        sincospif(x, &sn, &cs);
        s[i] = sn * (mag * sign);
        c[i] = cs * mag;
    }
    __syncwarp();
}
__device__ __forceinline__ void load_eight(const float *p, float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const float4 v = *reinterpret_cast<const float4 *>(p + 2 * i);
        f[i] = make_float2(v.x, v.y);
        f[i + 1] = make_float2(v.z, v.w);
    }
}

// A warp's ring of stages, each filled by bulk copies that its lane 0 starts and its own
// barrier counts.  Nobody else touches it.
template <int STAGES, int BYTES>
struct WarpRing {
    static constexpr int kStages = STAGES, kBytes = STAGES * BYTES;
    uint32_t bars, at;                // the barriers, and the stages, in shared memory
    unsigned issued = 0, used = 0;    // stages so far

    __device__ __forceinline__ WarpRing(const void *b, uint32_t stages) : bars(ptx::saddr(b)), at(stages) {}
    // by one thread, before the CTA's barrier
    static __device__ __forceinline__ void init(const void *b) {
        for (int s = 0; s < STAGES; ++s) ptx::mbar_init(ptx::saddr(b) + 8 * s, 1);
    }
    // the next stage: `bytes` of each of n sources (16-byte pieces), one behind the other
    template <int N>
    __device__ __forceinline__ void fill(int lane, const void *const (&src)[N], uint32_t bytes) {
        if (lane == 0) {
            const uint32_t bar = bars + 8 * (issued % STAGES), dst = at + issued % STAGES * BYTES;
            ptx::mbar_expect_tx(bar, N * bytes);
#pragma unroll
            for (int i = 0; i < N; ++i)
                asm volatile(
                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                        dst + i * (BYTES / N)),
                    "l"(src[i]), "r"(bytes), "r"(bar)
                    : "memory");
        }
        ++issued;
    }
    // waits for the oldest stage: its address, or 0 where the wait ran out
    __device__ __forceinline__ uint32_t wait(const ptx::Ctl &ctl) {
        const bool ok = __all_sync(0xffffffffu, ptx::wait_fast(bars + 8 * (used % STAGES), (used / STAGES) & 1, ctl));
        return ok ? at + used % STAGES * BYTES : 0;
    }
    // the oldest stage has been read by every lane
    __device__ __forceinline__ void release() {
        __syncwarp();
        ++used;
    }
    // copies in flight land before the CTA ends
    __device__ __forceinline__ void drain() {
        for (; used != issued; ++used)
            ptx::drain_bar(bars + 8 * (used % STAGES), (used / STAGES) & 1, kDefaultWaitLimit);
    }
};

// The eight pairs turned: pair i is (a[i], b[i]), or neighbours of a and then of b.
template <bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(float2 (&a)[4], float2 (&b)[4], const float2 (&c)[4],
                                           const float2 (&s)[4]) {
    if (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float2 &x = i < 4 ? a[i] : b[i - 4];
            const float cc = i & 1 ? c[i / 2].y : c[i / 2].x, ss = i & 1 ? s[i / 2].y : s[i / 2].x;
            x = make_float2(fmaf(x.x, cc, -x.y * ss), fmaf(x.y, cc, x.x * ss));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 u = ptx::ffma2(a[i], c[i], ptx::fmul2(minus(b[i]), s[i]));
            b[i] = ptx::ffma2(b[i], c[i], ptx::fmul2(a[i], s[i]));
            a[i] = u;
        }
    }
}

// 1 / sqrt(mean x^2 + eps) of the head whose values are on D / 16 neighbouring lanes.
// All lanes of the warp call it.
template <int D>
__device__ __forceinline__ float inverse_rms(const float2 (&a)[4], const float2 (&b)[4], float eps) {
    constexpr int LH = D / 16;
    auto squares = [&](float f) {
        float2 ss = make_float2(0.f, 0.f), tt = ss;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = f == 1.f ? a[i] : ptx::fmul2(a[i], both(f)), y = f == 1.f ? b[i] : ptx::fmul2(b[i], both(f));
            ss = ptx::ffma2(x, x, ss);
            tt = ptx::ffma2(y, y, tt);
        }
        float sum = (ss.x + ss.y) + (tt.x + tt.y);
#pragma unroll
        for (int o = 1; o < LH; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        return sum;
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
    return w32 ? static_cast<const float *>(w)[d] : __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[d]);
}

// a head over its root mean square, times the weights
template <int D>
__device__ __forceinline__ void normalise(float2 (&a)[4], float2 (&b)[4], const float2 (&wa)[4],
                                          const float2 (&wb)[4], float eps) {
    const float2 r = both(inverse_rms<D>(a, b, eps));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = ptx::fmul2(ptx::fmul2(a[i], r), wa[i]);
        b[i] = ptx::fmul2(ptx::fmul2(b[i], r), wb[i]);
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
