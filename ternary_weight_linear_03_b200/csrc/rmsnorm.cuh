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
// and r are read once, h and the codes written once (4096 x 8192 bf16 with a residual: 40.7 us,
// 5.8 TB/s of the 6.5 that a copy reaches; one row: 3.1 us, launch included).
#pragma once

#include "act_quant.cuh"
#include "common.cuh"

namespace bl {

constexpr float kFloatMax = 3.4028234663852886e38f;
constexpr int kNormMaxThreads = 1024;
constexpr int kNormMaxK = kNormMaxThreads * 4 * 8;  // a row is held by one block

// 8 elements as they are stored.
template <bool kBf16>
struct Raw8 {
  uint4 v[kBf16 ? 1 : 2];
};
template <bool kBf16, bool kStream = false>
__device__ __forceinline__ Raw8<kBf16> load_raw8(const void* row, int c) {
  Raw8<kBf16> r;
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
    const uint4* p = reinterpret_cast<const uint4*>(row) + (kBf16 ? 1 : 2) * c + i;
    r.v[i] = kStream ? ld_stream_v4(p) : *p;
  }
  return r;
}
template <bool kBf16>
__device__ __forceinline__ void store_raw8(void* row, int c, const Raw8<kBf16>& r) {
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); ++i) reinterpret_cast<uint4*>(row)[(kBf16 ? 1 : 2) * c + i] = r.v[i];
}
template <bool kBf16>
__device__ __forceinline__ void unpack8(const Raw8<kBf16>& r, float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (kBf16) {
      const uint32_t h = q == 0 ? r.v[0].x : q == 1 ? r.v[0].y : q == 2 ? r.v[0].z : r.v[0].w;
      v[2 * q] = __uint_as_float(h << 16);
      v[2 * q + 1] = __uint_as_float(h & 0xffff0000u);
    } else {
      const uint4& u = r.v[q >> 1];
      v[2 * q] = __uint_as_float((q & 1) ? u.z : u.x);
      v[2 * q + 1] = __uint_as_float((q & 1) ? u.w : u.y);
    }
  }
}
// The sum of two, rounded to the storage type.
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> add_raw8(const Raw8<kBf16>& a, const Raw8<kBf16>& b) {
  float x[8], y[8];
  unpack8<kBf16>(a, x);
  unpack8<kBf16>(b, y);
  uint32_t w[kBf16 ? 4 : 8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float u = __fadd_rn(x[2 * q], y[2 * q]), v = __fadd_rn(x[2 * q + 1], y[2 * q + 1]);
    if constexpr (kBf16) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(u, v);
      w[q] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      w[2 * q] = __float_as_uint(u);
      w[2 * q + 1] = __float_as_uint(v);
    }
  }
  Raw8<kBf16> r;
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); ++i) r.v[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  return r;
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

// quant_i8 of four values for an r that is finite and 127 / a rounded, |v| <= a: then |v r| is
// 127 at most after rounding, and adding 1.5 * 2^23 leaves the rounded code in the low byte.
// Half of quant_i8's instructions, none of them a conversion (4096 x 8192: 43.0 -> 40.8 us).
__device__ __forceinline__ uint32_t quant4(float a, float b, float c, float d, float r) {
  const float k = 12582912.0f;
  const uint32_t ta = __float_as_uint(__fadd_rn(__fmul_rn(a, r), k));
  const uint32_t tb = __float_as_uint(__fadd_rn(__fmul_rn(b, r), k));
  const uint32_t tc = __float_as_uint(__fadd_rn(__fmul_rn(c, r), k));
  const uint32_t td = __float_as_uint(__fadd_rn(__fmul_rn(d, r), k));
  return __byte_perm(__byte_perm(ta, tb, 0x0040), __byte_perm(tc, td, 0x0040), 0x5410);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}

__device__ __forceinline__ size_t row_offset(int t, int K, bool bf16) {
  return static_cast<size_t>(t) * static_cast<size_t>(K) * (bf16 ? 2 : 4);
}

// One block per row; thread i holds vectors i, i + blockDim.x, ... (V at most) of 8 elements, as
// stored (p is formed again from them for the codes: half the registers, twice the blocks).
// r, h, normed and rstd_out may be null; h may be x's or r's own memory (each thread reads its
// elements before it writes them).
template <bool kBf16, bool kWBf16, int V>
__global__ void __launch_bounds__(kNormMaxThreads) rmsnorm_quant_kernel(
    const void* x, const void* r, const void* __restrict__ w, float eps, int K,
    void* h, void* normed, int8_t* __restrict__ xq, float* __restrict__ scale,
    float* __restrict__ rstd_out) {
  __shared__ float red_s[32], red_m[32];
  grid_dependency_wait();
  allow_dependent_launch();  // a kernel that waits for this one may set itself up meanwhile
  const int t = blockIdx.x, T = blockDim.x, nv = K / 8;
  const size_t off = row_offset(t, K, kBf16);
  const char* xr = static_cast<const char*>(x) + off;
  const char* rr = r ? static_cast<const char*>(r) + off : nullptr;
  Raw8<kBf16> hv[V];
  float ss = 0.0f, m = 0.0f;
  // every load of the row before the first use (at V = 8 as far as 64 registers go)
#pragma unroll
  for (int v = 0; v < V; ++v) hv[v] = load_raw8<kBf16>(xr, min(v * T + static_cast<int>(threadIdx.x), nv - 1));
  if (rr) {
    Raw8<kBf16> b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = load_raw8<kBf16>(rr, min(v * T + static_cast<int>(threadIdx.x), nv - 1));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hv[v] = add_raw8<kBf16>(hv[v], b[v]);
      if (h && v * T + threadIdx.x < nv) store_raw8<kBf16>(static_cast<char*>(h) + off, v * T + threadIdx.x, hv[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * T + threadIdx.x;
    if (c < nv) {
      float p[8], g[8];
      unpack8<kBf16>(hv[v], p);
      load8<kWBf16>(w, c, g);
      float part = 0.0f;  // a thread adds sums of 8, not all of its 8 V squares in one row
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        part = fmaf(p[i], p[i], part);
        m = max_nan(m, fabsf(__fmul_rn(p[i], g[i])));  // a NaN of the gain is in p alone
      }
      ss = __fadd_rn(ss, part);
    }
  }
  ss = warp_sum(ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5;
  if (lane == 0) { red_s[warp] = ss; red_m[warp] = m; }
  __syncthreads();
  ss = warp_sum(lane < warps ? red_s[lane] : 0.0f);
  m = lane < warps ? red_m[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float rstd =
      __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(ss, static_cast<float>(K)), eps)));
  const float f = (m > 0.0f) ? __fdiv_rn(127.0f, m) : 0.0f;
  if (threadIdx.x == 0) {
    // NaN or infinite: x or the residual in either, the gain and the normalised row in top
    const float top = __fmul_rn(m, rstd);
    if (!(ss <= kFloatMax) || !(top <= kFloatMax)) record_status(kStatusNonfinite);
    scale[t] = (m > 0.0f) ? __fdiv_rn(top, 127.0f) : 0.0f;
    if (rstd_out) rstd_out[t] = rstd;
  }
  int8_t* qrow = xq + static_cast<size_t>(t) * K;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = v * T + threadIdx.x;
    if (c < nv) {
      float p[8], g[8];
      unpack8<kBf16>(hv[v], p);
      load8<kWBf16>(w, c, g);
      uint32_t q[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = __fmul_rn(p[i], g[i]);
      if (f <= kFloatMax) {
        q[0] = quant4(p[0], p[1], p[2], p[3], f);
        q[1] = quant4(p[4], p[5], p[6], p[7], f);
      } else {  // a subnormal maximum
#pragma unroll
        for (int i = 0; i < 8; ++i)
          q[i >> 2] |= (static_cast<uint32_t>(quant_i8(p[i], f)) & 0xffu) << (8 * (i & 3));
      }
      reinterpret_cast<uint2*>(qrow)[c] = make_uint2(q[0], q[1]);
      if (normed) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = __fmul_rn(p[i], rstd);
        store8<kBf16>(static_cast<char*>(normed) + off, c, p);
      }
    }
  }
}

// Gradient. With hat = h rstd and d = g w (g the gradient of the norm's output; the
// quantizer passes it straight through):
//   grad_x = grad_h + rstd (d - hat mean_k(d hat)),   grad_w[k] = sum_t g[t,k] hat[t,k]
// grad_x belongs to x and to the residual alike. Block b takes rows b, b + gridDim.x, ...; a
// thread keeps the same columns for all of them, so its part of grad_w stays in registers and is
// written once, to row b of part (summed over b by rmsnorm_grad_weight_kernel in a fixed
// order: no atomics, the same bits every time). Bound by memory: the next row's h and g are on
// their way while a row is reduced and written (one block of 512 threads fills an SM's
// registers, so nothing else would be; 4096 x 8192: 105 -> 58 us). Rows of more than 8192 are
// split over a cluster of cs blocks, which exchange their part of the row's sum.
constexpr int kNormBwdThreads = 512;
constexpr int kNormBwdMaxV = 2;
template <bool kHBf16, bool kGBf16, bool kOBf16, bool kWBf16, int V>
__global__ void __launch_bounds__(kNormBwdThreads) rmsnorm_backward_kernel(
    const void* __restrict__ g, const void* __restrict__ h, const void* __restrict__ w,
    const float* __restrict__ rstd, const void* grad_h, void* grad_x, float* __restrict__ part,
    int M, int K, int cs) {
  __shared__ float red[2][32];
  __shared__ float sum[2];
  const int T = blockDim.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = T >> 5;
  const int rank = cs > 1 ? static_cast<int>(cluster_rank()) : 0;
  // vectors of 8 columns [nv0, nv1) of this block
  const int each = (K / 8 + cs - 1) / cs, nv0 = min(rank * each, K / 8), nv1 = min(nv0 + each, K / 8);
  const int first = blockIdx.x / cs, stride = gridDim.x / cs;
  float dw[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[v][i] = 0.0f;
  auto at = [&](int v) { return nv0 + v * T + static_cast<int>(threadIdx.x); };
  auto column = [&](int v) { return max(min(at(v), nv1 - 1), 0); };
  Raw8<kHBf16> hn[V];
  Raw8<kGBf16> gn[V];
  auto fetch = [&](int t) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hn[v] = load_raw8<kHBf16>(static_cast<const char*>(h) + row_offset(t, K, kHBf16), column(v));
      gn[v] = load_raw8<kGBf16>(static_cast<const char*>(g) + row_offset(t, K, kGBf16), column(v));
    }
  };
  // hat, g and d of a vector
  auto values = [&](const Raw8<kHBf16>& hr, const Raw8<kGBf16>& gr, float rs, int v, float (&hat)[8],
                    float (&gv)[8], float (&d)[8]) {
    float wv[8];
    unpack8<kHBf16>(hr, hat);
    unpack8<kGBf16>(gr, gv);
    load8<kWBf16>(w, column(v), wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hat[i] = __fmul_rn(hat[i], rs);
      d[i] = __fmul_rn(gv[i], wv[i]);
    }
  };
  fetch(first);
  int turn = 0;
  for (int t = first; t < M; t += stride, turn ^= 1) {
    const size_t oo = row_offset(t, K, kOBf16);
    const float rs = rstd[t];
    Raw8<kHBf16> hc[V];
    Raw8<kGBf16> gc[V];
    Raw8<kOBf16> past[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      hc[v] = hn[v];
      gc[v] = gn[v];
      if (grad_h) past[v] = load_raw8<kOBf16>(static_cast<const char*>(grad_h) + oo, column(v));
    }
    fetch(min(t + stride, M - 1));
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float hat[8], gv[8], d[8];
      values(hc[v], gc[v], rs, v, hat, gv, d);
      if (at(v) < nv1) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dw[v][i] = fmaf(gv[i], hat[i], dw[v][i]);
          dot = fmaf(d[i], hat[i], dot);
        }
      }
    }
    dot = warp_sum(dot);
    if (lane == 0) red[turn][warp] = dot;
    __syncthreads();
    dot = warp_sum(lane < warps ? red[turn][lane] : 0.0f);
    if (cs > 1) {
      if (threadIdx.x == 0) sum[turn] = dot;
      cluster_barrier();
      dot = 0.0f;
      for (int k = 0; k < cs; ++k) dot += ld_cluster_f32(smem_u32(&sum[turn]), k);
    }
    const float mean = __fdiv_rn(dot, static_cast<float>(K));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (at(v) < nv1) {
        float hat[8], gv[8], d[8], o[8];
        values(hc[v], gc[v], rs, v, hat, gv, d);
        if (grad_h) {
          unpack8<kOBf16>(past[v], o);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = fmaf(rs, fmaf(-hat[i], mean, d[i]), o[i]);
        store8<kOBf16>(static_cast<char*>(grad_x) + oo, at(v), o);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (at(v) < nv1) store8<false>(part + static_cast<size_t>(first) * K, at(v), dw[v]);
  if (cs > 1) cluster_barrier();  // no block leaves while others read its sum
}

// grad_w[k] = sum_b part[b][k]. A block takes 32 columns; its 32 warps take rows b = w, w + 32,
// ... and are added in order.
constexpr int kNormGwThreads = 1024;
__global__ void __launch_bounds__(kNormGwThreads) rmsnorm_grad_weight_kernel(
    const float* __restrict__ part, int rows, int K, float* __restrict__ grad_w) {
  __shared__ float red[32][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int k = blockIdx.x * 32 + lane;  // K % 64 == 0: always inside
  float s = 0.0f;
  grid_dependency_wait();
#pragma unroll 8
  for (int b = warp; b < rows; b += 32) s += part[static_cast<size_t>(b) * K + k];
  red[warp][lane] = s;
  __syncthreads();
  s = warp_sum(red[lane][warp]);
  if (lane == 0) grad_w[blockIdx.x * 32 + warp] = s;
}

}  // namespace bl
