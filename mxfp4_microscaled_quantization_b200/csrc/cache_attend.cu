// cache_attend.cu -- single-token attention over the 8-bit paged cache.
//
// For sequence b, query head h (key head g = h / (Hq / Hkv)) and the cached
// tokens j < lens[b]:  s_j = scale q . (kc_j 2^ek),  o = sum_j e^(s_j - M)
// (vc_j 2^ev) / sum_j e^(s_j - M),  lse = M + ln sum_j e^(s_j - M), with the
// exponents of j's page.  lens[b] = 0 gives zeros and -inf.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.cuh"
#include "serve.cuh"

namespace mxattn {
namespace {

__device__ __forceinline__ void widen_e4m3x4(uint32_t w, float (&f)[4]) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w & 0xFFFFu)));
    widen2<true>(h2, f[0], f[1]);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(w >> 16)));
    widen2<true>(h2, f[2], f[3]);
}

// A warp per (sequence, query head).
template <int D, bool FP16>
__global__ void __launch_bounds__(32) cache_rows_kernel(const __grid_constant__ AttendArgs a) {
    constexpr int C = D / 32;
    const int b = blockIdx.x, h = blockIdx.y, lane = threadIdx.x;
    const int g = h / (a.Hq / a.Hkv), P = a.page_shift;
    int n = a.lens[b];
    const int64_t most = static_cast<int64_t>(a.max_pages) << P;
    if (n < 0 || n > most) {
        if (lane == 0) atomicOr(a.status, kStatusInvalid);
        n = n < 0 ? 0 : static_cast<int>(most);
    }
    const uint16_t* q = a.q + b * a.q_seq + h * a.q_head;
    float m = -INFINITY, l = 0.f, acc[C] = {};
    for (int j0 = 0; j0 < n; j0 += 32) {
        const int j = j0 + lane;
        float s = -INFINITY;
        int64_t row = -1;
        float vs = 0.f;
        if (j < n) {
            const int pg = a.table[static_cast<int64_t>(b) * a.table_stride + (j >> P)];
            if (pg >= 0 && pg < a.num_pages) {
                const int64_t cell = static_cast<int64_t>(pg) * a.Hkv + g;
                row = (cell << P) + (j & (a.page - 1));
                vs = exp2f(static_cast<float>(a.v_scales[cell]) - 127.f);
                float dot = 0.f;
                for (int c = 0; c < D; c += 4) {
                    float kf[4], q0, q1, q2, q3;
                    widen_e4m3x4(*reinterpret_cast<const uint32_t*>(a.k_codes + row * D + c), kf);
                    widen2<FP16>(*reinterpret_cast<const uint32_t*>(q + c), q0, q1);
                    widen2<FP16>(*reinterpret_cast<const uint32_t*>(q + c + 2), q2, q3);
                    dot = fmaf(kf[0], q0, fmaf(kf[1], q1, fmaf(kf[2], q2, fmaf(kf[3], q3, dot))));
                }
                s = dot * exp2f(static_cast<float>(a.k_scales[cell]) - 127.f) * a.scale;
            } else {
                atomicOr(a.status, kStatusInvalid);
            }
        }
        const float m_new = fmaxf(m, warp_max(s));
        const float base = m_new == -INFINITY ? 0.f : m_new;
        const float p = row >= 0 ? expf(s - base) : 0.f;
        const float alpha = expf(m - base);
        l = fmaf(l, alpha, warp_sum(p));
        for (int c = 0; c < C; ++c) acc[c] *= alpha;
        for (int i = 0; i < 32; ++i) {
            const float pi = __shfl_sync(0xffffffffu, p, i) * __shfl_sync(0xffffffffu, vs, i);
            const int64_t r = __shfl_sync(0xffffffffu, row, i);
            if (r < 0) continue;
            for (int c = 0; c < C; ++c) {
                float f[4];
                widen_e4m3x4(a.v_codes[r * D + lane * C + c], f);
                acc[c] = fmaf(pi, f[0], acc[c]);
            }
        }
        m = m_new;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    for (int c = 0; c < C; c += 2)
        *reinterpret_cast<uint32_t*>(a.o + b * a.o_seq + h * a.o_head + lane * C + c) = narrow2<FP16>(acc[c] * inv, acc[c + 1] * inv);
    if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(b) * a.Hq + h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t cache_attend_scratch_bytes(int, int, int) { return 0; }

cudaError_t launch_cache_attend(const AttendArgs& a, cudaStream_t stream) {
    if (a.B == 0) return cudaSuccess;
    const dim3 grid(a.B, a.Hq);
    if (a.d == 128) {
        if (a.fp16) cache_rows_kernel<128, true><<<grid, 32, 0, stream>>>(a);
        else cache_rows_kernel<128, false><<<grid, 32, 0, stream>>>(a);
    } else {
        if (a.fp16) cache_rows_kernel<64, true><<<grid, 32, 0, stream>>>(a);
        else cache_rows_kernel<64, false><<<grid, 32, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace mxattn
