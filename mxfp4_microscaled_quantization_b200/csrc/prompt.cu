// prompt.cu -- attention over packed prompts of different lengths (16-bit
// operands, grouped heads, causal or not).
//
// For sequence b with n queries and m keys, query i and head h (key head g = h
// / (Hq / Hkv)):  s_ij = scale q_i . k_j over the keys j it sees (causal: j <=
// i + m - n, the queries being the newest n tokens),  o_i = sum_j e^(s_ij - M)
// v_j / sum_j e^(s_ij - M),  lse_i = M + ln sum_j e^(s_ij - M).  A row that
// sees no key gives zeros and -inf.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.cuh"
#include "serve.cuh"

namespace mxattn {
namespace {

// A warp per (query row, head).
template <int D, bool FP16>
__global__ void __launch_bounds__(128) prompt_rows_kernel(const __grid_constant__ PromptArgs a) {
    const int row = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5);
    if (h >= a.Hq) return;
    for (int b = 0; b < a.B; ++b) {
        int q0, q1, k0, k1;
        bool ok = packed_range(a.q_offsets, b, a.total_q, q0, q1);
        ok &= packed_range(a.kv_offsets, b, a.total_kv, k0, k1);
        if (!ok && threadIdx.x == 0) atomicOr(a.status, kStatusInvalid);
        if (row < q0 || row >= q1) continue;
        const int m = k1 - k0;
        const int n = a.causal ? max(0, min(m, row - q0 + 1 + m - (q1 - q0))) : m;
        const int g = h / (a.Hq / a.Hkv);
        attend_row<D, FP16>(a.q + row * a.q_token + h * a.q_head, a.k + k0 * a.k_token + g * a.k_head,
                            a.v + k0 * a.v_token + g * a.v_head, a.k_token, a.v_token, n, a.scale,
                            a.o + row * a.o_token + h * a.o_head,
                            a.lse == nullptr ? nullptr : a.lse + h * a.lse_head + row);
        return;
    }
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs& a, cudaStream_t stream) {
    if (a.total_q == 0) return cudaSuccess;
    const dim3 grid(static_cast<unsigned>(a.total_q), (a.Hq + 3) / 4);
    if (a.d == 128) {
        if (a.fp16) prompt_rows_kernel<128, true><<<grid, 128, 0, stream>>>(a);
        else prompt_rows_kernel<128, false><<<grid, 128, 0, stream>>>(a);
    } else {
        if (a.fp16) prompt_rows_kernel<64, true><<<grid, 128, 0, stream>>>(a);
        else prompt_rows_kernel<64, false><<<grid, 128, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace mxattn
