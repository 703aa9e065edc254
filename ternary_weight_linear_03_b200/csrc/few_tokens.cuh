// The ternary x int8 contraction for a few tokens, on warp-level int8 matrix instructions.
//
// A warp takes 16 weight rows as the 16 x 32 operand (unsigned codes u = c + 1) and 8 tokens
// as the 32 x 8 operand of m16n8k32; sum_k u q - sum_k q = sum_k c q as in the other kernels.
// The order of k inside a product is free as long as both operands use the same one, so the
// fragments are taken as the packed format has them: lane (g, t) = (lane / 4, lane % 4) loads
// 16 bytes (64 trits) of rows g and g + 8; plane j of each 4-byte word is one register of the
// weight fragment (one mask), and the 4 codes that belong to it, 4 consecutive
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
// column 8 n + g that belong to word i of them. acc[j][n]: rows g (0, 1) and g + 8 (2, 3), columns
// 8 n + 2 t and 8 n + 2 t + 1 of the products with fragment j. The masks are what bounds this
// (the logic pipe takes a warp's instruction in two cycles), so the planes stay where they
// are in the word and an accumulator per plane takes the factor 4^j.
//   kFour: fragment j is plane j, (w & 3 4^j); a column is a token. 4 masks a word.
//   kPairs, for up to 4 tokens, which leave half of the 8 columns empty: fragment j is planes
//     0 .. j, w & (4^(j+1) - 1), so the last is the word itself and needs no mask. With P_j the
//     products of fragment j, plane j is (P_j - P_(j-1)) / 4^j: an even column holds the token's
//     codes of plane j, the odd one behind it those of plane j + 1, to be subtracted.
//     3 masks a word (70B up, one token, from shifted planes: 15.2 -> 13.2 us).
//   kTwo, where 16 columns leave no registers for four accumulators: planes 2 and 3 are shifted
//     onto 0 and 1. 4 masks and a shift a word, but half as much to clear and to add up
//     (70B down, 16 tokens: 23.7 -> 22.3 us; 64 tokens of 8 wide experts: 137 -> 122 us).
enum PlaneMode : int { kFour = 0, kPairs = 1, kTwo = 2 };
__host__ __device__ constexpr int planes(int mode) { return mode == kTwo ? 2 : 4; }

template <int NT, int MODE>
__device__ __forceinline__ void ternary_step(int (&acc)[planes(MODE)][NT][4], const uint4& wa,
                                             const uint4& wb, const uint4 (&q)[NT][4]) {
#pragma unroll
  for (int i = 0; i < 4; i += 2)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t m = MODE == kPairs ? (j == 3 ? 0xffffffffu : ((4u << (2 * j)) - 1u) * 0x01010101u)
                         : MODE == kTwo ? 0x03030303u << (2 * (j & 1))
                                        : 0x03030303u << (2 * j);
      const int sh = (MODE == kTwo && j > 1) ? 4 : 0;
      const uint32_t a0 = (word_of(wa, i) >> sh) & m, a1 = (word_of(wb, i) >> sh) & m;
      const uint32_t a2 = (word_of(wa, i + 1) >> sh) & m, a3 = (word_of(wb, i + 1) >> sh) & m;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        mma_u8s8(acc[MODE == kTwo ? j & 1 : j][n], a0, a1, a2, a3, word_of(q[n][i], j), word_of(q[n][i + 1], j));
    }
}
// The exact sum: of column e & 1, or (kPairs) of the token of both columns (e even).
template <int NT, int MODE>
__device__ __forceinline__ int ternary_sum(const int (&acc)[planes(MODE)][NT][4], int n, int e) {
  if constexpr (MODE == kPairs)
    return acc[0][n][e] + ((acc[1][n][e] - acc[0][n][e + 1]) >> 2) +
           ((acc[2][n][e] - acc[1][n][e + 1]) >> 4) + ((acc[3][n][e] - acc[2][n][e + 1]) >> 6);
  else if constexpr (MODE == kTwo)
    return acc[0][n][e] + (acc[1][n][e] >> 2);
  else
    return acc[0][n][e] + (acc[1][n][e] >> 2) + (acc[2][n][e] >> 4) + (acc[3][n][e] >> 6);
}
// Clears the sums, minus[n] (the negative sum of codes) for the columns that u = c + 1 wants
// it taken off: in kPairs the even ones.
template <int NT, int MODE>
__device__ __forceinline__ void ternary_clear(int (&acc)[planes(MODE)][NT][4], const int (&minus)[NT][2]) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc[0][n][e] = minus[n][e & 1];
#pragma unroll
      for (int j = 1; j < planes(MODE); ++j) acc[j][n][e] = 0;
    }
}
// minus[] from each lane's sum of the codes it loaded for token n (of column 8 n + g, or
// (kPairs) column g).
template <int MODE>
__device__ __forceinline__ void minus_of(int sum, int (&minus)[2]) {
  const int t4 = threadIdx.x & 3;
  sum += __shfl_xor_sync(0xffffffffu, sum, 1);
  sum += __shfl_xor_sync(0xffffffffu, sum, 2);
  minus[0] = -__shfl_sync(0xffffffffu, sum, 8 * t4);
  minus[1] = -__shfl_sync(0xffffffffu, sum, 8 * t4 + 4);
  if (MODE == kPairs) minus[1] = 0;
}
__device__ __forceinline__ int dot_ones(const uint4& v, int sum) {
#pragma unroll
  for (int j = 0; j < 4; ++j) sum = __dp4a(static_cast<int>(word_of(v, j)), 0x01010101, sum);
  return sum;
}
// Adds a tile's sums of this warp to those of its block, to[row of the tile][column], for the
// columns below `valid`.
template <int NT, int MODE>
__device__ __forceinline__ void ternary_add(const int (&acc)[planes(MODE)][NT][4], int* to, int valid) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; e += MODE == kPairs ? 2 : 1) {
      const int t = MODE == kPairs ? t4 : 8 * n + 2 * t4 + (e & 1);
      if (t < valid) atomicAdd(to + (g + (e < 2 ? 0 : 8)) * 8 * NT + t, ternary_sum<NT, MODE>(acc, n, e));
    }
}
// Codes of an odd column in kPairs: those of the plane behind, none behind the last.
__device__ __forceinline__ uint4 next_plane(const uint4& v) { return make_uint4(v.y, v.z, v.w, 0u); }

constexpr int kFewMaxWarps = 8;     // warps of a block
constexpr int kFewMaxCluster = 8;
constexpr int kFewRound = 32;       // tiles of 16 rows between two joins of the sums
// 256-trit steps of 16 rows (1 KB) that a warp keeps in flight: two blocks of 8 warps and their
// sums fill the shared memory of an SM.
__host__ __device__ constexpr int few_depth(int NT) { return NT == 1 ? 12 : 8; }
// Steps of a warp: as many as its registers hold codes for (fewer steps per warp mean more
// sums to join for the same weights: one token, 70B up, 1 / 2 / 4 steps: 17.8 / 15.8 / 13.9 us).
__host__ __device__ constexpr int few_steps(int NT) { return 4 / NT; }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most `kPending` of this thread's groups are in flight.
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// The 16 bytes at shared address `addr` of this block, in block `rank` of the cluster.
__device__ __forceinline__ int4 ld_cluster_v4(uint32_t addr, uint32_t rank) {
  uint32_t a;
  int4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// One stage of transpose4: the lanes that differ in bit `mask` exchange b of the one without
// the bit for a of the one with it.
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b, bool has, int mask) {
  const uint32_t got = __shfl_xor_sync(0xffffffffu, has ? a : b, mask);
  a = has ? got : a;
  b = has ? b : got;
}
__device__ __forceinline__ void exchange(uint4& a, uint4& b, bool has, int mask) {
  exchange(a.x, b.x, has, mask);
  exchange(a.y, b.y, has, mask);
  exchange(a.z, b.z, has, mask);
  exchange(a.w, b.w, has, mask);
}
// v[i] of lane t and v[t] of lane i change places within each four lanes (t = lane % 4).
__device__ __forceinline__ void transpose4(uint4 (&v)[4], int t) {
  exchange(v[0], v[2], t & 2, 2);
  exchange(v[1], v[3], t & 2, 2);
  exchange(v[0], v[1], t & 1, 1);
  exchange(v[2], v[3], t & 1, 1);
}

// y[t,n] = fl(float(sum_k c q) fl(scale_t gamma)) for M <= 8 NT tokens (4 in kPairs).
// Bound by the packed weights' bytes up to 8 tokens (70B up, 28672 x 8192: 13.2 us at one token,
// 14.8 at eight; 4.4 TB/s with launch and prologue, the loop itself runs at the memory's pace),
// by the matrix instructions' share beyond (20.3 us at sixteen; 70B down 22.3 us).
// K is split over all warps of a cluster of blocks, few_steps steps of 256 to one, so that a
// warp can keep its part of every token in registers for the whole kernel: the codes are
// read once per cluster, not once per block (every block asks for the same lines, and with all
// of them staged in every block's shared memory 8 tokens of 8192 x 8192 took 15.5 us instead of
// 7.0), and the loop has no shared-memory reads of codes. Each warp then streams its columns of
// the cluster's row tiles through a ring of its own in shared memory (a lane reads back what it
// copied itself, so nobody else is waited for), and adds a tile's integer sums to the block's
// (exact in any order): no warp waits for another before the join. The ring holds what the
// memory delivers while the codes arrive. The stream has no bounds to check: rows past N and
// chunks past K read the last ones, and meet outputs that are not written and codes that are
// zero. Nothing is read ahead of the wait for the kernel before, which may be the one that wrote
// the weights (reading them ahead would save 1.3 us).
template <int NT, int MODE, bool kOBf16>
__global__ void __launch_bounds__(32 * kFewMaxWarps, 2) few_tokens_kernel(
    const int8_t* __restrict__ xq, const float* __restrict__ scale, const uint8_t* __restrict__ packed,
    const float* __restrict__ gamma_ptr, void* __restrict__ y, int M, int N, int K, int cs) {
  constexpr int S = few_steps(NT);
  constexpr int kAhead = few_depth(NT) / S;  // tiles whose weights are in flight
  extern __shared__ __align__(16) uint8_t ring_all[];  // [warp][tile][step][row half][lane] 16 bytes
  __shared__ __align__(16) int sums[kFewRound * 16 * 8 * NT];  // [row of the round][token]
  __shared__ float factor[8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int warps = blockDim.x >> 5;
  const uint32_t rank = cs > 1 ? cluster_rank() : 0u;
  const int chunks = K / 64;
  const int c = 4 * S * (static_cast<int>(rank) * warps + warp) + t4;  // this lane's chunks: c, c + 4, ...
  // 16-row tiles first, first + clusters, ...: `count` of them
  const int tiles = (N + 15) / 16, clusters = gridDim.x / cs, first = blockIdx.x / cs;
  const int count = (tiles - first + clusters - 1) / clusters;
  const size_t pitch = static_cast<size_t>(K / 4);
  const uint32_t ring = smem_u32(ring_all) + warp * kAhead * S * 1024 + lane * 16;
  auto fetch = [&](uint32_t slot, int i) {
    if (i < count) {
      const int row = (first + i * clusters) * 16 + g;
      const uint8_t* a = packed + min(row, N - 1) * pitch;
      const uint8_t* b = packed + min(row + 8, N - 1) * pitch;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int at = 16 * min(c + 4 * s, chunks - 1);
        cp_async16(slot + s * 1024, a + at);
        cp_async16(slot + s * 1024 + 512, b + at);
      }
    }
    cp_async_commit();
  };
  for (int i = threadIdx.x; i < kFewRound * 32 * NT; i += blockDim.x)
    reinterpret_cast<uint4*>(sums)[i] = make_uint4(0u, 0u, 0u, 0u);
  // the kernel before may have written the weights too: nothing is read ahead of this wait
  grid_dependency_wait();
#pragma unroll
  for (int r = 0; r < kAhead; ++r) fetch(ring + r * S * 1024, r);
  uint4 q[S][NT][4];
  int minus[NT][2];  // -sum of the warp's codes of the tokens of this lane's columns
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = MODE == kPairs ? g >> 1 : 8 * n + g;
    const uint4* row = reinterpret_cast<const uint4*>(xq + static_cast<size_t>(min(t, M - 1)) * K);
    int sum = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      // Lane t needs the four 16-byte units of chunk c + 4 s. With more than 8 tokens the lanes
      // of a row read neighbouring units (a request then touches 8 lines, not 16) and exchange
      // them (16 tokens, 70B up / down: 22.9 / 27.9 -> 20.7 / 23.6 us; 8 tokens, up: 14.9 -> 15.6).
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int chunk = NT == 1 ? c + 4 * s : c - t4 + 4 * s + i, unit = NT == 1 ? i : t4;
        v[i] = (t < M && chunk < chunks) ? row[4 * chunk + unit] : make_uint4(0u, 0u, 0u, 0u);
      }
      if (NT > 1) transpose4(v, t4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum = dot_ones(v[i], sum);
        q[s][n][i] = MODE == kPairs && (g & 1) ? next_plane(v[i]) : v[i];
      }
    }
    minus_of<MODE>(sum, minus[n]);
  }
  if (threadIdx.x < M) factor[threadIdx.x] = __fmul_rn(scale[threadIdx.x], *gamma_ptr);
  __syncthreads();  // the sums are zero
  uint32_t slot = ring;
  for (int i0 = 0; i0 < count; i0 += kFewRound) {
    const int i1 = min(count, i0 + kFewRound);
    for (int i = i0; i < i1; ++i) {
      int acc[planes(MODE)][NT][4];
      ternary_clear<NT, MODE>(acc, minus);
      cp_async_wait<kAhead - 1>();
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const uint4 wa = ld_shared_v4(slot + s * 1024), wb = ld_shared_v4(slot + s * 1024 + 512);
        ternary_step<NT, MODE>(acc, wa, wb, q[s]);
      }
      fetch(slot, i + kAhead);
      slot = slot + S * 1024 == ring + kAhead * S * 1024 ? ring : slot + S * 1024;
      ternary_add<NT, MODE>(acc, sums + (i - i0) * 16 * 8 * NT, M);
    }
    if (cs > 1) cluster_barrier(); else __syncthreads();
    // The cluster's blocks share the tiles of the round; a thread takes four tokens of a row.
    const int share = (i1 - i0 - static_cast<int>(rank) + cs - 1) / cs, quads = (M + 3) / 4;
    for (int u = threadIdx.x; u < share * quads * 16; u += blockDim.x) {
      const int r = u & 15, at = (u >> 4) / quads, t0 = 4 * ((u >> 4) - at * quads);
      const int i = i0 + static_cast<int>(rank) + at * cs, row = (first + i * clusters) * 16 + r;
      const int* from = sums + ((i - i0) * 16 + r) * 8 * NT + t0;
      int sum[4] = {};
      if (cs > 1) {
#pragma unroll 4
        for (int k = 0; k < cs; ++k) {
          const int4 v = ld_cluster_v4(smem_u32(from), k);
          sum[0] += v.x; sum[1] += v.y; sum[2] += v.z; sum[3] += v.w;
        }
      } else {
        const int4 v = *reinterpret_cast<const int4*>(from);
        sum[0] = v.x; sum[1] = v.y; sum[2] = v.z; sum[3] = v.w;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = t0 + e;
        if (t < M && row < N) {
          const float v = __fmul_rn(__int2float_rn(sum[e]), factor[t]);
          const size_t to = static_cast<size_t>(t) * N + row;
          if (kOBf16) static_cast<__nv_bfloat16*>(y)[to] = __float2bfloat16_rn(v);
          else static_cast<float*>(y)[to] = v;
        }
      }
    }
    if (cs > 1) cluster_barrier(); else __syncthreads();  // nobody reads these sums any more
    if (i1 < count) {
      for (int i = threadIdx.x; i < kFewRound * 32 * NT; i += blockDim.x)
        reinterpret_cast<uint4*>(sums)[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
    }
  }
}

}  // namespace bl
