// move_rows.cu -- rows between token order and expert order.
//
//   permute    rows[inv[t,k]] = x[t] for every slot with a position, x in
//              bf16 or restored from E4M3 codes and their per-128 scales
//   unpermute  out[t] = bf16( sum over k ascending of y[inv[t,k]] + residual[t] )
// Each is the other's transpose, so each is also the other's gradient.  Both
// go token by token: permute reads a token's row once and writes it K times,
// unpermute reads its K rows and writes one.
#include "common.cuh"
#include "internal.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint4 restore_bf16x8(const uint2 q, float scale) {
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t word = i < 2 ? q.x : q.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * (i & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// One thread per (token, 8 columns).
template <bool FP8>
__global__ void __launch_bounds__(kThreads) permute_rows_kernel(
    const void *__restrict__ x, const float *__restrict__ x_scale, const int32_t *__restrict__ inv,
    const float *__restrict__ weights, int64_t T, int K, int V, int n_out, uint4 *__restrict__ out,
    float *__restrict__ row_weights) {
    const int64_t n = T * V;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / V;
        const int c = (int)(i - t * V);
        const uint4 v = FP8 ? restore_bf16x8(__ldg(static_cast<const uint2 *>(x) + i), __ldg(x_scale + t * (V / 16) + c / 16))
                            : __ldg(static_cast<const uint4 *>(x) + i);
        for (int k = 0; k < K; ++k) {
            const int p = __ldg(inv + t * K + k);
            if (p < 0 || p >= n_out) continue;
            out[(int64_t)p * V + c] = v;
            if (c == 0 && row_weights) row_weights[p] = __ldg(weights + t * K + k);
        }
    }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads) unpermute_rows_kernel(
    const void *__restrict__ y, const int32_t *__restrict__ inv, const uint4 *__restrict__ residual,
    const float *__restrict__ drow, int64_t T, int K, int V, int n_in, uint4 *__restrict__ out,
    float *__restrict__ dweights) {
    const int64_t n = T * V;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / V;
        const int c = (int)(i - t * V);
        float acc[8] = {};
        for (int k = 0; k < K; ++k) {
            const int p = __ldg(inv + t * K + k);
            const bool on = p >= 0 && p < n_in;
            if (c == 0 && dweights) dweights[t * K + k] = on ? __ldg(drow + p) : 0.0f;
            if (!on) continue;
            float f[8];
            if (F32) {
                const float4 *q = static_cast<const float4 *>(y) + ((int64_t)p * V + c) * 2;
                const float4 a = __ldg(q), b = __ldg(q + 1);
                f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
                f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            } else {
                unpack_bf16x8(__ldg(static_cast<const uint4 *>(y) + (int64_t)p * V + c), f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += f[j];
        }
        if (residual) {
            float f[8];
            unpack_bf16x8(__ldg(residual + i), f);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] += f[j];
        }
        out[i] = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                            pack_bf16x2(acc[6], acc[7]));
    }
}

dim3 grid_of(int64_t n) {
    return dim3((unsigned)std::min<int64_t>((n + kThreads - 1) / kThreads, 16LL * num_sms()));
}

}  // namespace

cudaError_t launch_permute_rows(const void *x, const float *x_scale, const int32_t *inv, const float *weights,
                                int64_t T, int K, int H, int n_out, void *out, float *row_weights, cudaStream_t st) {
    auto *kernel = x_scale ? permute_rows_kernel<true> : permute_rows_kernel<false>;
    return launch_k(kernel, grid_of(T * (H / 8)), dim3(kThreads), 0, st, false, x, x_scale, inv, weights, T, K, H / 8,
                    n_out, (uint4 *)out, row_weights);
}

cudaError_t launch_unpermute_rows(const void *y, bool y_fp32, const int32_t *inv, const void *residual,
                                  const float *drow, int64_t T, int K, int H, int n_in, void *out, float *dweights,
                                  cudaStream_t st) {
    auto *kernel = y_fp32 ? unpermute_rows_kernel<true> : unpermute_rows_kernel<false>;
    return launch_k(kernel, grid_of(T * (H / 8)), dim3(kThreads), 0, st, false, y, inv, (const uint4 *)residual, drow,
                    T, K, H / 8, n_in, (uint4 *)out, dweights);
}

}  // namespace moe
