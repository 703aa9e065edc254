// A mixture-of-experts layer with ternary experts, for a few tokens:
//   logits[t,e] = sum_d x[t,d] R[e,d];  S_t = the top_k largest (ties: the lowest expert)
//   w[t,e] = softmax of the logits, over all experts or (renormalize) over S_t
//   q, s = the int8 codes and scale of x_t;  G = gate, U = up, D = down of expert e in S_t
//   i[t,e] = act(G(q, s)) * U(q, s),  y_t = sum_{e in S_t} w[t,e] D(codes of i[t,e])
// A pair p = t top_k + s is slot s of token t.
#pragma once

#include "few_tokens.cuh"
#include "rmsnorm.cuh"

namespace bl {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeThreads = 128;

enum MoeAct : int { kActSilu = 0, kActRelu2 = 1 };

__device__ __forceinline__ float moe_act(float g, int act) {
  if (act == kActSilu) return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g)));
  const float r = fmaxf(g, 0.0f);
  return __fmul_rn(r, r);
}

// A float's bits as an unsigned number that orders like the float; NaN below everything.
// Never 0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v == v)) return 1u;
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Top-k of a token's logits by one warp: lane l holds logits l, l + 32, ...
__device__ __forceinline__ void moe_top_k(const float* logits, int E, int top_k, bool renorm,
                                          int* __restrict__ ids, float* __restrict__ weights) {
  constexpr int kPer = kMoeMaxExperts / 32;
  const int lane = threadIdx.x & 31;
  uint32_t key[kPer];
  uint32_t best = 0u;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = 32 * i + lane;
    const float v = e < E ? logits[e] : 0.0f;
    bad |= !(fabsf(v) <= kFloatMax);
    key[i] = e < E ? order_key(v) : 0u;
    best = max(best, key[i]);
  }
  if (bad) record_status(kStatusNonfinite);
  float top = 0.0f, sum = 0.0f, mine = 0.0f;
  int mine_e = 0;
  for (int s = 0; s < top_k; ++s) {
    const uint32_t k = __reduce_max_sync(0xffffffffu, best);
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int i = kPer - 1; i >= 0; --i)
      if (key[i] == k) e = 32 * i + lane;
    e = __reduce_min_sync(0xffffffffu, e);
    const float v = logits[e];
    if (s == 0) top = v;
    const float p = expf(v - top);
    if (lane == s) { mine = p; mine_e = static_cast<int>(e); }
    if (renorm) sum += p;
    best = 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (32u * i + lane == e) key[i] = 0u;
      best = max(best, key[i]);
    }
  }
  if (!renorm) {
    for (int e = lane; e < E; e += 32) sum += expf(logits[e] - top);
    sum = warp_sum(sum);
  }
  if (lane < top_k) {
    ids[lane] = mine_e;
    weights[lane] = __fdiv_rn(mine, sum);
  }
}

// Logits and choice of one token per block, a warp per expert in turn.
template <bool kXBf16>
__global__ void __launch_bounds__(256) moe_route_kernel(
    const void* __restrict__ x, const void* __restrict__ router, int r_bf16, int D, int E, int top_k,
    int renorm, int* __restrict__ ids, float* __restrict__ weights) {
  __shared__ float logits[kMoeMaxExperts];
  const int t = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const char* xr = static_cast<const char*>(x) + row_offset(t, D, kXBf16);
  for (int e = warp; e < E; e += 8) {
    const char* rr = static_cast<const char*>(router) + row_offset(e, D, r_bf16);
    float s = 0.0f;
    for (int c = lane; c < D / 8; c += 32) {
      float a[8], b[8];
      load8<kXBf16>(xr, c, a);
      load8_any(rr, r_bf16, c, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = fmaf(a[i], b[i], s);
    }
    s = warp_sum(s);
    if (lane == 0) logits[e] = s;
  }
  __syncthreads();
  if (warp == 0) moe_top_k(logits, E, top_k, renorm, ids + t * top_k, weights + t * top_k);
}

// The pairs of one expert, in order, into list; their number. Called by a whole block.
__device__ __forceinline__ int moe_pairs_of(const int* __restrict__ ids, int pairs, int expert,
                                            int* list, int* count) {
  if (threadIdx.x < 32) {
    int n = 0;
    for (int p0 = 0; p0 < pairs; p0 += 32) {
      const int p = p0 + static_cast<int>(threadIdx.x);
      const bool is = p < pairs && ids[p] == expert;
      const uint32_t b = __ballot_sync(0xffffffffu, is);
      if (is) list[n + __popc(b & ((1u << threadIdx.x) - 1u))] = p;
      n += __popc(b);
    }
    if (threadIdx.x == 0) *count = n;
  }
  __syncthreads();
  return *count;
}

// One 16-row tile of `rows` against up to 8 pairs of codes (pair list[i0 + g] reads row
// list[...] / div of q).
__device__ __forceinline__ void moe_tile(int (&acc)[4][1][4], const uint8_t* __restrict__ w, int row0,
                                         int K, const int8_t* __restrict__ q, const int8_t* qrow) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3, chunks = K / 64;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  const uint4* pa = reinterpret_cast<const uint4*>(w + static_cast<size_t>(row0 + g) * (K / 4));
  const uint4* pb = reinterpret_cast<const uint4*>(w + static_cast<size_t>(row0 + g + 8) * (K / 4));
  for (int c = t4; c - t4 < chunks; c += 4) {
    const bool in = c < chunks;
    const uint4 wa = in ? ld_stream_v4(pa + c) : zero, wb = in ? ld_stream_v4(pb + c) : zero;
    uint4 v[1][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[0][i] = (in && qrow) ? reinterpret_cast<const uint4*>(qrow)[4 * c + i] : zero;
    ternary_step<1, false>(acc, wa, wb, v);
  }
}

// inner[p][f] = act(G) * U for the pairs of expert blockIdx.y; a warp per 16 rows.
__global__ void __launch_bounds__(kMoeThreads) moe_gate_up_kernel(
    const int* __restrict__ ids, const int8_t* __restrict__ xq, const float* __restrict__ xscale,
    const int* __restrict__ xsum, const uint8_t* __restrict__ gate, const uint8_t* __restrict__ up,
    const float* __restrict__ gate_gamma, const float* __restrict__ up_gamma, int pairs, int top_k,
    int D, int F, int act, float* __restrict__ inner) {
  __shared__ int list[kMoeMaxTokens];
  __shared__ int count;
  const int e = blockIdx.y;
  const int n = moe_pairs_of(ids, pairs, e, list, &count);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int row0 = (blockIdx.x * (kMoeThreads / 32) + warp) * 16;
  if (row0 >= F) return;
  const size_t per = static_cast<size_t>(F) * (D / 4);
  const float gg = gate_gamma[e], gu = up_gamma[e];
  for (int i0 = 0; i0 < n; i0 += 8) {
    const int8_t* qrow = i0 + g < n ? xq + static_cast<size_t>(list[i0 + g] / top_k) * D : nullptr;
    int ag[4][1][4] = {}, au[4][1][4] = {};
    moe_tile(ag, gate + e * per, row0, D, xq, qrow);
    moe_tile(au, up + e * per, row0, D, xq, qrow);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 2 * t4 + (j & 1);
      if (i < n) {
        const int p = list[i], t = p / top_k;
        const float s = xscale[t];
        const float G = __fmul_rn(__int2float_rn(ternary_sum<1, false>(ag, 0, j) - xsum[t]), __fmul_rn(s, gg));
        const float U = __fmul_rn(__int2float_rn(ternary_sum<1, false>(au, 0, j) - xsum[t]), __fmul_rn(s, gu));
        inner[static_cast<size_t>(p) * F + row0 + g + (j < 2 ? 0 : 8)] = __fmul_rn(moe_act(G, act), U);
      }
    }
  }
}

// part[p][d] = the down projection of pair p.
__global__ void __launch_bounds__(kMoeThreads) moe_down_kernel(
    const int* __restrict__ ids, const int8_t* __restrict__ hq, const float* __restrict__ hscale,
    const int* __restrict__ hsum, const uint8_t* __restrict__ down, const float* __restrict__ down_gamma,
    int pairs, int D, int F, float* __restrict__ part) {
  __shared__ int list[kMoeMaxTokens];
  __shared__ int count;
  const int e = blockIdx.y;
  const int n = moe_pairs_of(ids, pairs, e, list, &count);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int row0 = (blockIdx.x * (kMoeThreads / 32) + warp) * 16;
  if (row0 >= D) return;
  const float gd = down_gamma[e];
  for (int i0 = 0; i0 < n; i0 += 8) {
    const int8_t* qrow = i0 + g < n ? hq + static_cast<size_t>(list[i0 + g]) * F : nullptr;
    int acc[4][1][4] = {};
    moe_tile(acc, down + e * (static_cast<size_t>(D) * (F / 4)), row0, F, hq, qrow);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + 2 * t4 + (j & 1);
      if (i < n) {
        const int p = list[i];
        part[static_cast<size_t>(p) * D + row0 + g + (j < 2 ? 0 : 8)] =
            __fmul_rn(__int2float_rn(ternary_sum<1, false>(acc, 0, j) - hsum[p]), __fmul_rn(hscale[p], gd));
      }
    }
  }
}

// y_t = sum_s w[t,s] part[t top_k + s], in the order of the slots.
template <bool kOBf16>
__global__ void __launch_bounds__(256) moe_combine_kernel(const float* __restrict__ part,
                                                         const float* __restrict__ weights, int D,
                                                         int top_k, void* __restrict__ y) {
  const int t = blockIdx.y, d = blockIdx.x * 256 + threadIdx.x;
  if (d >= D) return;
  float s = 0.0f;
  for (int k = 0; k < top_k; ++k)
    s = fmaf(weights[t * top_k + k], part[static_cast<size_t>(t * top_k + k) * D + d], s);
  const size_t at = static_cast<size_t>(t) * D + d;
  if (kOBf16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(s);
  else static_cast<float*>(y)[at] = s;
}

}  // namespace bl
