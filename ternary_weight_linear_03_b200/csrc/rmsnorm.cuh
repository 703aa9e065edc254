// Root-mean-square norm that adds the residual and quantizes its output to int8, and the
// gradient of the norm.
//
//   h = rnd(x + r),  rstd = 1 / sqrt(mean_k h^2 + eps),  n = h rstd w
//   p = fl(h w),  a = max_k |p|,  q = clip(rne(fl(p fl(127/a))), -127, 127)
//   scale = fl(fl(a rstd) / 127)
//
// rstd is one positive factor per row, so it cancels out of the codes: max |n| = rstd a and
// n / max |n| = p / a. Both row statistics (the sum of squares and a) are therefore taken in
// the same pass over the registers that hold the row, and one block barrier joins them; x
// and r are read once, h and the codes written once.
#pragma once

#include "act_quant.cuh"
#include "common.cuh"

namespace bl {

constexpr float kFloatMax = 3.4028234663852886e38f;
constexpr int kNormMaxV = 4;                              // 8-element vectors per thread, at most
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxK = kNormMaxThreads * kNormMaxV * 8;  // a row is held by one block

// Rounds to the storage type and back.
template <bool kBf16>
__device__ __forceinline__ float round_to(float v) {
  return kBf16 ? __bfloat162float(__float2bfloat16_rn(v)) : v;
}

template <bool kBf16>
__device__ __forceinline__ void store8(void* row, int c, const float (&v)[8]) {
  if (kBf16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    reinterpret_cast<uint4*>(row)[c] = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(row)[2 * c] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(row)[2 * c + 1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

__device__ __forceinline__ void load8_any(const void* row, bool bf16, int c, float (&v)[8]) {
  if (bf16) load8<true>(row, c, v); else load8<false>(row, c, v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ size_t row_offset(int t, int K, bool bf16) {
  return static_cast<size_t>(t) * static_cast<size_t>(K) * (bf16 ? 2 : 4);
}

// One block per row; thread i holds vectors i, i + blockDim.x, ... (V at most) of 8 elements.
// r, h, normed and rstd_out may be null; h may be x's or r's own memory (each thread reads its
// elements before it writes them).
template <bool kBf16, int V>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_quant_kernel(
    const void* x, const void* r, const void* __restrict__ w, int w_bf16, float eps, int K,
    void* h, void* normed, int8_t* __restrict__ xq, float* __restrict__ scale,
    float* __restrict__ rstd_out) {
  __shared__ float red_s[32], red_m[32];
  const int t = blockIdx.x, T = blockDim.x, nv = K / 8;
  const size_t off = row_offset(t, K, kBf16);
  const char* xr = static_cast<const char*>(x) + off;
  const char* rr = r ? static_cast<const char*>(r) + off : nullptr;
  float p[V][8];
  float ss = 0.0f, m = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * T + threadIdx.x;
    if (c < nv) {
      load8<kBf16>(xr, c, p[v]);
      if (rr) {
        float b[8];
        load8<kBf16>(rr, c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) p[v][i] = round_to<kBf16>(__fadd_rn(p[v][i], b[i]));
        if (h) store8<kBf16>(static_cast<char*>(h) + off, c, p[v]);
      }
      float g[8];
      load8_any(w, w_bf16, c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(p[v][i], p[v][i], ss);
        p[v][i] = __fmul_rn(p[v][i], g[i]);
        m = fmaxf(m, fabsf(p[v][i]));
      }
    }
  }
  ss = warp_sum(ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5;
  if (lane == 0) { red_s[warp] = ss; red_m[warp] = m; }
  __syncthreads();
  ss = warp_sum(lane < warps ? red_s[lane] : 0.0f);
  m = lane < warps ? red_m[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float rstd =
      __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps)));
  const float f = (m > 0.0f) ? __fdiv_rn(127.0f, m) : 0.0f;
  if (threadIdx.x == 0) {
    // NaN never wins fmaxf, but reaches the sum of squares
    if (!(ss <= kFloatMax) || !(m <= kFloatMax)) record_status(kStatusNonfinite);
    scale[t] = (m > 0.0f) ? __fdiv_rn(__fmul_rn(m, rstd), 127.0f) : 0.0f;
    if (rstd_out) rstd_out[t] = rstd;
  }
  int8_t* qrow = xq + static_cast<size_t>(t) * K;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * T + threadIdx.x;
    if (c < nv) {
      uint32_t q[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i >> 2] |= (static_cast<uint32_t>(quant_i8(p[v][i], f)) & 0xffu) << (8 * (i & 3));
      reinterpret_cast<uint2*>(qrow)[c] = make_uint2(q[0], q[1]);
      if (normed) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[v][i] = __fmul_rn(p[v][i], rstd);
        store8<kBf16>(static_cast<char*>(normed) + off, c, p[v]);
      }
    }
  }
}

// Gradient. With hat = h rstd and d = g w (g the gradient of the norm's output; the
// quantizer passes it straight through):
//   grad_x = grad_h + rstd (d - hat mean_k(d hat)),   grad_w[k] = sum_t g[t,k] hat[t,k]
// grad_x belongs to x and to the residual alike. Block b takes rows b, b + gridDim.x, ...;
// a thread keeps the same columns for all of them, so its part of grad_w stays in
// registers and is written once, to row b of part (summed over b by
// rmsnorm_grad_weight_kernel in a fixed order: no atomics, the same bits every time).
// Rows of more than 512 x V vectors leave 64 registers a thread: kReload reads h and g again
// (from L1/L2) for the second half instead of keeping them.
template <bool kHBf16, bool kGBf16, bool kOBf16, int V, bool kReload>
__global__ void __launch_bounds__(kReload ? kNormMaxThreads : kNormMaxThreads / 2) rmsnorm_backward_kernel(
    const void* __restrict__ g, const void* __restrict__ h, const void* __restrict__ w, int w_bf16,
    const float* __restrict__ rstd, const void* grad_h, void* grad_x, float* __restrict__ part,
    int M, int K) {
  __shared__ float red[32];
  const int T = blockDim.x, nv = K / 8;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5;
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
  for (int t = blockIdx.x; t < M; t += gridDim.x) {
    const char* hr = static_cast<const char*>(h) + row_offset(t, K, kHBf16);
    const char* gr = static_cast<const char*>(g) + row_offset(t, K, kGBf16);
    const size_t oo = row_offset(t, K, kOBf16);
    const float rs = rstd[t];
    constexpr int kKeep = kReload ? 1 : V;
    float hat[kKeep][8], d[kKeep][8];
    float dot = 0.0f;
    auto take = [&](int c, float (&ht)[8], float (&dv)[8], bool first, float (&sum)[8]) {
      float wv[8];
      load8<kHBf16>(hr, c, ht);
      load8<kGBf16>(gr, c, dv);
      load8_any(w, w_bf16, c, wv);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ht[i] = __fmul_rn(ht[i], rs);
        if (first) sum[i] = fmaf(dv[i], ht[i], sum[i]);
        dv[i] = __fmul_rn(dv[i], wv[i]);
        if (first) dot = fmaf(dv[i], ht[i], dot);
      }
    };
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * T + threadIdx.x, i = kReload ? 0 : v;
      if (c < nv) take(c, hat[i], d[i], true, dw[v]);
    }
    dot = warp_sum(dot);
    if (lane == 0) red[warp] = dot;
    __syncthreads();
    dot = warp_sum(lane < warps ? red[lane] : 0.0f);
    __syncthreads();  // red is written again for the next row
    const float mean = __fdiv_rn(dot, static_cast<float>(K));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = v * T + threadIdx.x, iv = kReload ? 0 : v;
      if (c < nv) {
        float o[8];
        if (kReload) take(c, hat[0], d[0], false, dw[v]);
        if (grad_h) {
          load8<kOBf16>(static_cast<const char*>(grad_h) + oo, c, o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = fmaf(rs, fmaf(-hat[iv][i], mean, d[iv][i]), o[i]);
        store8<kOBf16>(static_cast<char*>(grad_x) + oo, c, o);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * T + threadIdx.x;
    if (c < nv) store8<false>(part + static_cast<size_t>(blockIdx.x) * K, c, dw[v]);
  }
}

// grad_w[k] = sum_b part[b][k]. A block takes 32 columns; its 8 warps take rows b = w, w + 8,
// ... and are added in order.
constexpr int kNormGwThreads = 256;
__global__ void __launch_bounds__(kNormGwThreads) rmsnorm_grad_weight_kernel(
    const float* __restrict__ part, int rows, int K, float* __restrict__ grad_w) {
  __shared__ float red[8][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = blockIdx.x * 32 + lane;  // K % 64 == 0: always inside
  float s = 0.0f;
  for (int b = warp; b < rows; b += 8) s += part[static_cast<size_t>(b) * K + k];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    grad_w[k] = s;
  }
}

}  // namespace bl
