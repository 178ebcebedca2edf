// serve.cuh -- what the serving operators share: 16-bit input types, batch
// offsets read on the device, the exact evaluation of one attention row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "ptx.cuh"

namespace mxattn {

constexpr uint32_t kStatusInvalid = 1u;  // MXATTN_ERR_INVALID: an offset, length or page index out of range
constexpr uint32_t kStatusTimeout = 4u;  // MXATTN_ERR_TIMEOUT

// The two 16-bit input and output types: widening is exact, narrowing rounds
// to nearest even (the result's own type: the one rounding of an output).
template <bool FP16>
__device__ __forceinline__ void widen2(uint32_t w, float& lo, float& hi) {
    if constexpr (FP16) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w);
        lo = __low2float(h);
        hi = __high2float(h);
    } else {
        lo = __uint_as_float(w << 16);
        hi = __uint_as_float(w & 0xFFFF0000u);
    }
}
template <bool FP16>
__device__ __forceinline__ uint32_t narrow2(float lo, float hi) {
    uint32_t w;
    if constexpr (FP16)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// Smallest e with amax <= 448 * 2^e for amax >= 0 in fp32 (448 = 1.75 * 2^8):
// floor(log2 amax) - 8, plus one where the significand exceeds 1.75.  amax = 0
// gives -127; fp16's subnormals are normal numbers in fp32, and bf16's end at
// the clamp.
__device__ __forceinline__ int e4m3_exponent(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    const int E = static_cast<int>(bits >> 23);
    if (E == 0) return -127;
    const int e = E - 135 + (((bits & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
    return min(max(e, -127), 127);
}

// Two fp32 values to two E4M3 codes (lo in the low byte): nearest even, beyond
// +-448 saturated, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ void unpack_e4m3x2(uint32_t b, float& lo, float& hi) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(b)));
    widen2<true>(h2, lo, hi);
}

// Sequence b's rows [begin, end) from the offsets of a packed batch.  Offsets
// that decrease or leave [0, total] are brought into range, so no access can
// leave the tensors, and reported.
__device__ __forceinline__ bool packed_range(const int32_t* offsets, int b, int64_t total, int& begin, int& end) {
    const int o0 = offsets[b], o1 = offsets[b + 1];
    const int t = static_cast<int>(total);
    begin = min(max(o0, 0), t);
    end = min(max(o1, begin), t);
    return begin == o0 && end == o1;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One attention row, o = softmax(q K^T scale) V over keys 0 .. n - 1, by one
// warp in fp32: a lane per key for the scores, a lane per D / 32 channels for
// the sum over V.  No key behind n is read, so nothing that a row may not see
// reaches it.  k and v: row 0 of the keys, strides in elements.  Writes o, or
// with `part` instead channel c, in fp32, to part[(c / 4) * 512 + c % 4].
template <int D, bool FP16>
__device__ __noinline__ void attend_row(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t k_stride,
                                        int64_t v_stride, int n, float scale, uint16_t* o, float* part) {
    constexpr int C = D / 32;  // channels of a lane
    const int lane = threadIdx.x & 31;
    float m = -INFINITY, l = 0.f, acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        if (j < n) {
            const uint16_t* kr = k + j * k_stride;
            float dot = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 8) {
                const uint4 a = *reinterpret_cast<const uint4*>(q + c), b = *reinterpret_cast<const uint4*>(kr + c);
                const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float a0, a1, b0, b1;
                    widen2<FP16>(aw[i], a0, a1);
                    widen2<FP16>(bw[i], b0, b1);
                    dot = fmaf(a0, b0, fmaf(a1, b1, dot));
                }
            }
            s = dot * scale;
        }
        const float m_new = fmaxf(m, warp_max(s));
        const float base = isinf(m_new) && m_new < 0.f ? 0.f : m_new;
        const float p = j < n ? expf(s - base) : 0.f;
        const float alpha = expf(m - base);
        l = fmaf(l, alpha, warp_sum(p));
#pragma unroll
        for (int c = 0; c < C; ++c) acc[c] *= alpha;
        for (int i = 0; i < min(32, n - j0); ++i) {
            const float pi = __shfl_sync(0xffffffffu, p, i);
            const uint16_t* vr = v + (j0 + i) * v_stride + lane * C;
#pragma unroll
            for (int c = 0; c < C; c += 2) {
                float v0, v1;
                widen2<FP16>(*reinterpret_cast<const uint32_t*>(vr + c), v0, v1);
                acc[c] = fmaf(pi, v0, acc[c]);
                acc[c + 1] = fmaf(pi, v1, acc[c + 1]);
            }
        }
        m = m_new;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing: zeros, lse -inf
    if (part != nullptr) {
#pragma unroll
        for (int c = 0; c < C; ++c) part[(lane * C + c) / 4 * 512 + (lane * C + c) % 4] = acc[c] * inv;
        return;
    }
#pragma unroll
    for (int c = 0; c < C; c += 2)
        *reinterpret_cast<uint32_t*>(o + lane * C + c) = narrow2<FP16>(acc[c] * inv, acc[c + 1] * inv);
}

}  // namespace mxattn
