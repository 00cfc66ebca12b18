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

// Rows to process: the device's count when there is one, within the buffers.
__device__ __forceinline__ int64_t live_rows(const int32_t *n_rows, int rows) {
    return n_rows ? min(max(__ldg(n_rows), 0), rows) : rows;
}

// Half a warp per block of 128 features (gate and up), 8 values a lane; the
// half-warps stride over the (row, block) pairs, stepping both parts of the
// index (a 64-bit division per pair cost a quarter of the kernel).
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_kernel(
    const uint4 *__restrict__ gu, const float *__restrict__ weight, const int32_t *__restrict__ n_rows, int rows,
    int F, uint4 *__restrict__ h, uint2 *__restrict__ codes, float *__restrict__ scale) {
    pdl_wait();
    pdl_launch_dependents();
    const int NB = F / 128, V = F / 8, sub = threadIdx.x & 15;
    const int64_t live = live_rows(n_rows, rows);
    const int64_t first = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 4;
    const int64_t stride = ((int64_t)gridDim.x * kThreads) >> 4;
    const int64_t step_r = stride / NB;
    const int step_b = (int)(stride - step_r * NB);
    int64_t r = first / NB;
    int b = (int)(first - r * NB);
    // the two halves of a warp stay together: the block scale is found by warp shuffles
    while (__any_sync(0xFFFFFFFFu, r < live)) {
        const bool on = r < live;
        const int64_t at = r * 2 * V + b * 16 + sub;
        const uint4 vg = on ? __ldg(gu + at) : make_uint4(0, 0, 0, 0);
        const uint4 vu = on ? __ldg(gu + at + V) : make_uint4(0, 0, 0, 0);
        const float p = weight && on ? __ldg(weight + r) : 1.0f;
        float g[8], u[8], o[8];
        unpack_bf16x8(vg, g);
        unpack_bf16x8(vu, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = p * (g[i] * sigmoid_f(g[i]) * u[i]);
        float sg, su;
        const uint2 qg = checkpoint8(g, sg), qu = checkpoint8(u, su);
        if (on) {
            h[r * V + b * 16 + sub] = pack_bf16x8(o);
            codes[at] = qg;
            codes[at + V] = qu;
            if (sub < 2) scale[r * 2 * NB + sub * NB + b] = sub ? su : sg;
        }
        r += step_r;
        b += step_b;
        if (b >= NB) {
            b -= NB;
            ++r;
        }
    }
}

// WPR warps per row: one for many rows, four for few (the row's loads then
// all go out at once).
template <int WPR>
__global__ void __launch_bounds__(kThreads) swiglu_checkpoint_backward_kernel(
    const uint2 *__restrict__ codes, const float *__restrict__ scale, const uint4 *__restrict__ dh,
    const float *__restrict__ weight, const int32_t *__restrict__ n_rows, int rows, int F, uint4 *__restrict__ dgu,
    uint4 *__restrict__ h, float *__restrict__ dweight) {
    __shared__ float s_dot[kThreads / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int NB = F / 128, V = F / 8, lane = lane_id(), warp = threadIdx.x >> 5;
    const int64_t live = live_rows(n_rows, rows);
    const int64_t stride = (int64_t)gridDim.x * (kThreads / 32 / WPR);
    for (int64_t r0 = (int64_t)blockIdx.x * (kThreads / 32 / WPR); r0 < live; r0 += stride) {
        const int64_t r = r0 + warp / WPR;
        float dot = 0.f;
        if (r < live) {
            const float p = weight ? __ldg(weight + r) : 1.0f;
            const uint2 *cr = codes + r * 2 * V;
            const float *sr = scale + r * 2 * NB;
            const uint4 *dr = dh + r * V;
            uint4 *gr = dgu + r * 2 * V, *hr = h ? h + r * V : nullptr;
#pragma unroll 2
            for (int c = (warp % WPR) * 32 + lane; c < V; c += 32 * WPR) {
                float g[8], u[8], d[8], dg[8], du[8], o[8];
                restore8_e4m3(__ldg(cr + c), __ldg(sr + c / 16), g);
                restore8_e4m3(__ldg(cr + V + c), __ldg(sr + NB + c / 16), u);
                unpack_bf16x8(__ldg(dr + c), d);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = sigmoid_f(g[i]), a = g[i] * s, pd = p * d[i], au = a * u[i];
                    dot += d[i] * au;
                    o[i] = p * au;
                    dg[i] = pd * u[i] * (s + a * (1.0f - s));
                    du[i] = pd * a;
                }
                gr[c] = pack_bf16x8(dg);
                gr[V + c] = pack_bf16x8(du);
                if (hr) hr[c] = pack_bf16x8(o);
            }
        }
        if (dweight) {
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
            if (WPR == 1) {
                if (lane == 0 && r < live) dweight[r] = dot;
            } else {
                if (lane == 0) s_dot[warp] = dot;
                __syncthreads();
                if (lane == 0 && warp % WPR == 0 && r < live) {
                    float sum = s_dot[warp];
                    for (int i = 1; i < WPR; ++i) sum += s_dot[warp + i];
                    dweight[r] = sum;
                }
                __syncthreads();
            }
        }
    }
}

}  // namespace

cudaError_t launch_swiglu_checkpoint(const void *gu, const float *weight, const int32_t *n_rows, int rows, int F,
                                     void *h, void *codes, float *scale, cudaStream_t st) {
    const int64_t blocks = ((int64_t)rows * (F / 8) + kThreads - 1) / kThreads;
    return launch_k(swiglu_checkpoint_kernel, dim3((unsigned)std::min<int64_t>(blocks, 8LL * num_sms())),
                    dim3(kThreads), 0, st, true, (const uint4 *)gu, weight, n_rows, rows, F, (uint4 *)h,
                    (uint2 *)codes, scale);
}

cudaError_t launch_swiglu_checkpoint_backward(const void *codes, const float *scale, const void *dh,
                                              const float *weight, const int32_t *n_rows, int rows, int F, void *dgu,
                                              void *h, float *dweight, cudaStream_t st) {
    const bool few = rows <= 8 * num_sms();
    const int per_block = kThreads / 32 / (few ? 4 : 1);
    const int64_t blocks = ((int64_t)rows + per_block - 1) / per_block;
    auto *kernel = few ? swiglu_checkpoint_backward_kernel<4> : swiglu_checkpoint_backward_kernel<1>;
    return launch_k(kernel, dim3((unsigned)std::min<int64_t>(blocks, 8LL * num_sms())), dim3(kThreads), 0, st, true,
                    (const uint2 *)codes, scale, (const uint4 *)dh, weight, n_rows, rows, F, (uint4 *)dgu, (uint4 *)h,
                    dweight);
}

}  // namespace moe
