// swiglu_checkpoint.cu -- the experts' SwiGLU for training: the forward pass
// keeps its gate and up activations in 8 bits (E4M3 codes, one power-of-two
// scale per 128 values: the rule of quantize_fp8_block128), the backward pass
// recomputes everything it needs from them.
//
// With g, u the two halves of a row, s = sigmoid(g), a = g s, p the row's
// router weight:
//   forward    h = p a u                            from the bf16 g, u
//   backward   h = p a u, dp = sum_f dh a u,        from the restored g, u
//              dg = p dh u (s + a (1 - s)), du = p dh a
// Since h carries p, dh (the gradient of the down product's input before p)
// gives p's gradient by one dot product per row and the expert output need
// not be kept.
#include <float.h>

#include "common.cuh"
#include "internal.h"

#include <algorithm>

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid_f(float g) { return __fdividef(1.0f, 1.0f + expf(-g)); }

// Block scale and codes of 8 values per lane, 16 lanes per block of 128, as
// quant8_e4m3; a block that holds an infinity takes the exponent of the
// largest finite value, whose largest code is restored as an infinity (448 *
// 2^120 overflows), and a NaN keeps its own code.
__device__ __forceinline__ uint2 checkpoint8(const float (&f)[8], float &scale) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const int k = fp8_block_exp(fminf(amax, FLT_MAX));
    const float inv = pow2f(-k);
    scale = pow2f(k);
    uint2 q;
    q.x = (uint32_t)e4m3x2(f[0] * inv, f[1] * inv) | ((uint32_t)e4m3x2(f[2] * inv, f[3] * inv) << 16);
    q.y = (uint32_t)e4m3x2(f[4] * inv, f[5] * inv) | ((uint32_t)e4m3x2(f[6] * inv, f[7] * inv) << 16);
    return q;
}

__device__ __forceinline__ void restore8(const uint2 q, float scale, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t word = i < 2 ? q.x : q.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * (i & 1))), __NV_E4M3);
        const float2 v = __half22float2(__half2(h));
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Rows to process: the device's count when there is one, within the buffers.
__device__ __forceinline__ int64_t live_rows(const int32_t *n_rows, int rows) {
    return n_rows ? min(max(__ldg(n_rows), 0), rows) : rows;
}

// One lane per 8 features of a row.
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_kernel(
    const uint4 *__restrict__ gu, const float *__restrict__ weight, const int32_t *__restrict__ n_rows, int rows,
    int F, uint4 *__restrict__ h, uint2 *__restrict__ codes, float *__restrict__ scale) {
    const int V = F / 8;
    const int64_t n = live_rows(n_rows, rows) * V;
    for (int64_t v0 = (int64_t)blockIdx.x * kThreads; v0 < n; v0 += (int64_t)gridDim.x * kThreads) {
        const int64_t v = v0 + threadIdx.x;
        const bool on = v < n;
        const int64_t r = on ? v / V : 0;
        const int c = on ? (int)(v - r * V) : 0;
        float g[8], u[8], o[8];
        unpack_bf16x8(on ? __ldg(gu + r * 2 * V + c) : make_uint4(0, 0, 0, 0), g);
        unpack_bf16x8(on ? __ldg(gu + r * 2 * V + V + c) : make_uint4(0, 0, 0, 0), u);
        const float p = weight && on ? __ldg(weight + r) : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = p * (g[i] * sigmoid_f(g[i]) * u[i]);
        float sg, su;
        const uint2 qg = checkpoint8(g, sg), qu = checkpoint8(u, su);   // every lane of the warp takes part
        if (on) {
            h[r * V + c] = pack8(o);
            codes[r * 2 * V + c] = qg;
            codes[r * 2 * V + V + c] = qu;
            if ((c & 15) == 0) {
                scale[r * (2 * V / 16) + c / 16] = sg;
                scale[r * (2 * V / 16) + V / 16 + c / 16] = su;
            }
        }
    }
}

// One warp per row.
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_backward_kernel(
    const uint2 *__restrict__ codes, const float *__restrict__ scale, const uint4 *__restrict__ dh,
    const float *__restrict__ weight, const int32_t *__restrict__ n_rows, int rows, int F, uint4 *__restrict__ dgu,
    uint4 *__restrict__ h, float *__restrict__ dweight) {
    const int V = F / 8, lane = lane_id();
    const int64_t n = live_rows(n_rows, rows);
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); r < n;
         r += (int64_t)gridDim.x * (kThreads / 32)) {
        const float p = weight ? __ldg(weight + r) : 1.0f;
        float dot = 0.f;
        for (int c = lane; c < V; c += 32) {
            float g[8], u[8], d[8], dg[8], du[8], o[8];
            restore8(__ldg(codes + r * 2 * V + c), __ldg(scale + r * (2 * V / 16) + c / 16), g);
            restore8(__ldg(codes + r * 2 * V + V + c), __ldg(scale + r * (2 * V / 16) + (V + c) / 16), u);
            unpack_bf16x8(__ldg(dh + r * V + c), d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid_f(g[i]), a = g[i] * s, pd = p * d[i];
                dot += d[i] * (a * u[i]);
                o[i] = p * (a * u[i]);
                dg[i] = pd * u[i] * (s + a * (1.0f - s));
                du[i] = pd * a;
            }
            dgu[r * 2 * V + c] = pack8(dg);
            dgu[r * 2 * V + V + c] = pack8(du);
            if (h) h[r * V + c] = pack8(o);
        }
        if (dweight) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            if (lane == 0) dweight[r] = dot;
        }
    }
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const void *gu, const float *weight, const int32_t *n_rows, int rows, int F,
                                     void *h, void *codes, float *scale, cudaStream_t st) {
    const int64_t blocks = ((int64_t)rows * (F / 8) + kThreads - 1) / kThreads;
    return launch_k(swiglu_checkpoint_kernel, dim3((unsigned)std::min<int64_t>(blocks, 8LL * num_sms())),
                    dim3(kThreads), 0, st, false, (const uint4 *)gu, weight, n_rows, rows, F, (uint4 *)h,
                    (uint2 *)codes, scale);
}

cudaError_t launch_swiglu_checkpoint_backward(const void *codes, const float *scale, const void *dh,
                                              const float *weight, const int32_t *n_rows, int rows, int F, void *dgu,
                                              void *h, float *dweight, cudaStream_t st) {
    const int64_t blocks = ((int64_t)rows + kThreads / 32 - 1) / (kThreads / 32);
    return launch_k(swiglu_checkpoint_backward_kernel, dim3((unsigned)std::min<int64_t>(blocks, 8LL * num_sms())),
                    dim3(kThreads), 0, st, false, (const uint2 *)codes, scale, (const uint4 *)dh, weight, n_rows, rows,
                    F, (uint4 *)dgu, (uint4 *)h, dweight);
}

}  // namespace moe
