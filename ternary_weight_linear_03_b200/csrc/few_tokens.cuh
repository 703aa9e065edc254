// The ternary x int8 contraction for a few tokens, on warp-level int8 matrix instructions.
//
// A warp takes 16 weight rows as the 16 x 32 operand (unsigned codes u = c + 1) and 8 tokens
// as the 32 x 8 operand of m16n8k32; sum_k u q - sum_k q = sum_k c q as in the other kernels.
// The order of k inside a product is free as long as both operands use the same one, so the
// fragments are taken as the packed format has them: lane (g, t) = (lane / 4, lane % 4) loads
// 16 bytes (64 trits) of rows g and g + 8; plane j of each 4-byte word is one register of the
// weight fragment (a shift and a mask), and the 4 codes that belong to it, 4 consecutive
// bytes of token g, one register of the token fragment. Four lanes cover 256 trits.
#pragma once

#include "act_quant.cuh"
#include "common.cuh"

namespace bl {

// D (16 x 8, int32) += A (16 x 32, unsigned bytes) B (32 x 8, signed bytes).
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// 256 trits of 16 rows: wa, wb the lane's 16 bytes of rows g and g + 8, q[n][i] the 16 codes of
// token 8 n + g that belong to word i of them. acc[n]: rows g (0, 1) and g + 8 (2, 3), tokens
// 8 n + 2 t and 8 n + 2 t + 1.
template <int NT>
__device__ __forceinline__ void ternary_step(int (&acc)[NT][4], const uint4& wa, const uint4& wb,
                                             const uint4 (&q)[NT][4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a0 = (word_of(wa, i) >> (2 * j)) & 0x03030303u;
      const uint32_t a1 = (word_of(wb, i) >> (2 * j)) & 0x03030303u;
      const uint32_t a2 = (word_of(wa, i + 1) >> (2 * j)) & 0x03030303u;
      const uint32_t a3 = (word_of(wb, i + 1) >> (2 * j)) & 0x03030303u;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma_u8s8(acc[n], a0, a1, a2, a3, word_of(q[n][i], j), word_of(q[n][i + 1], j));
    }
}

constexpr int kFewThreads = 128;

// y[t,n] = fl(float(acc) fl(scale_t gamma)) for M <= 8 NT tokens: a warp per 16 rows of the
// packed weights, token codes straight from global memory.
template <int NT, bool kOBf16>
__global__ void __launch_bounds__(kFewThreads) few_tokens_kernel(
    const int8_t* __restrict__ xq, const float* __restrict__ scale, const uint8_t* __restrict__ packed,
    const float* __restrict__ gamma_ptr, void* __restrict__ y, int M, int N, int K) {
  __shared__ int rowsum[8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  for (int t = warp; t < M; t += kFewThreads / 32) {
    const uint4* row = reinterpret_cast<const uint4*>(xq + static_cast<size_t>(t) * K);
    int s = 0;
    for (int c = lane; c < K / 16; c += 32) {
      const uint4 v = row[c];
#pragma unroll
      for (int i = 0; i < 4; ++i) s = __dp4a(static_cast<int>(word_of(v, i)), 0x01010101, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) rowsum[t] = s;
  }
  __syncthreads();
  const int row0 = (blockIdx.x * (kFewThreads / 32) + warp) * 16;
  if (row0 >= N) return;
  const int chunks = K / 64;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const int ra = row0 + g, rb = row0 + g + 8;
  const uint4* pa = reinterpret_cast<const uint4*>(packed + static_cast<size_t>(ra) * (K / 4));
  const uint4* pb = reinterpret_cast<const uint4*>(packed + static_cast<size_t>(rb) * (K / 4));
  int acc[NT][4] = {};
  for (int c = t4; c - t4 < chunks; c += 4) {
    const bool in = c < chunks;
    const uint4 wa = (in && ra < N) ? ld_stream_v4(pa + c) : zero;
    const uint4 wb = (in && rb < N) ? ld_stream_v4(pb + c) : zero;
    uint4 q[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int t = 8 * n + g;
      const uint4* px = reinterpret_cast<const uint4*>(xq + static_cast<size_t>(t) * K);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[n][i] = (in && t < M) ? px[4 * c + i] : zero;
    }
    ternary_step<NT>(acc, wa, wb, q);
  }
  const float gamma = *gamma_ptr;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int t = 8 * n + 2 * t4 + (e & 1), r = (e < 2) ? ra : rb;
      if (t < M && r < N) {
        const float v = __fmul_rn(__int2float_rn(acc[n][e] - rowsum[t]), __fmul_rn(scale[t], gamma));
        const size_t at = static_cast<size_t>(t) * N + r;
        if (kOBf16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(v);
        else static_cast<float*>(y)[at] = v;
      }
    }
}

}  // namespace bl
