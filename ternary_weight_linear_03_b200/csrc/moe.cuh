// A mixture-of-experts layer with ternary experts, for a few tokens:
//   logits[t,e] = sum_d x[t,d] R[e,d];  S_t = the top_k largest (ties: the lowest expert)
//   w[t,e] = softmax of the logits, over all experts or (renormalize) over S_t
//   q, s = the int8 codes and scale of x_t;  G = gate, U = up, D = down of expert e in S_t
//   i[t,e] = act(G(q, s)) * U(q, s),  y_t = sum_{e in S_t} w[t,e] D(codes of i[t,e])
// A pair p = t top_k + s is slot s of token t.
#pragma once

#include <type_traits>

#include "few_tokens.cuh"
#include "rmsnorm.cuh"

namespace bl {

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxWidth = 16384;  // of x and of an expert

enum MoeAct : int { kActSilu = 0, kActRelu2 = 1 };

__device__ __forceinline__ float moe_act(float g, int act) {
  if (act == kActSilu) return __fdiv_rn(g, __fadd_rn(1.0f, expf(-g)));
  const float r = max_nan(g, 0.0f);
  return __fmul_rn(r, r);
}

// A float's bits as an unsigned number that orders like the float; NaN below everything.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v == v)) return 1u;
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.0f));  // -0 as +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// The choice among a token's E logits (shared memory) by a block of kThreads >= E threads, a
// power of two: an expert's rank is the number of those before it, which as many lanes count as
// there are threads for an expert (rounds of maxima, or one thread per expert, are chains of
// thousands of cycles on a single warp). keys, chosen: shared memory for E and top_k words.
template <int kThreads>
__device__ __forceinline__ void moe_top_k(const float* logits, int E, int top_k, bool renorm, uint32_t* keys,
                                          int* chosen, int* __restrict__ ids, float* __restrict__ weights) {
  const int tid = threadIdx.x;
  if (tid < E) {
    const float mine = logits[tid];
    if (!(fabsf(mine) <= kFloatMax)) record_status(kStatusNonfinite);
    keys[tid] = order_key(mine);
  }
  __syncthreads();
  int share = 1;  // lanes to an expert
  while (share < 32 && 2 * share * E <= kThreads) share *= 2;
  const int e = tid / share;
  int rank = 0;
  if (e < E) {
    const uint32_t key = keys[e];
#pragma unroll 4
    for (int i = tid % share; i < E; i += share) rank += keys[i] > key || (keys[i] == key && i < e);
  }
  for (int o = 1; o < share; o *= 2) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (e < E && tid % share == 0 && rank < top_k) chosen[rank] = e;
  __syncthreads();
  if (tid >= 32) return;
  const float top = logits[chosen[0]];
  const float mine = tid < top_k ? expf(logits[chosen[tid]] - top) : 0.0f;
  float sum = mine;
  if (!renorm) {
    sum = 0.0f;
    for (int i = tid; i < E; i += 32) sum += expf(logits[i] - top);
  }
  sum = warp_sum(sum);
  if (tid < top_k) {
    ids[tid] = chosen[tid];
    weights[tid] = __fdiv_rn(mine, sum);
  }
}

// ------------------------------------------------------------------------------- route
// One cluster of `blocks` blocks (8, or 2 when there are more tokens than eighths of the GPU) per
// token. Each block takes its share of the experts' logits and of the row's codes, and the
// first one, to whose shared memory the others send theirs, chooses. Also clears what the next
// kernels add to. A dot product is the sum of `share` warps' parts, in order, and a part that of
// 32 lanes' vectors; share follows from E alone, so a token's logits, and with them its experts,
// have the same bits whatever other tokens there are. Bound by latency, so all of the router is
// asked for at once: share is what spreads the experts over all warps of 8 blocks, with eight
// vectors of the router in flight per lane (64 experts of 4096, one token: 17 -> 10 thousand
// cycles with the choice in one pass of ranks).
constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;

template <bool kXBf16, bool kRBf16>
__global__ void __launch_bounds__(kRouteThreads, 1) moe_route_kernel(
    const void* __restrict__ x, const void* __restrict__ router, int D, int E, int top_k, int renorm,
    int* __restrict__ ids, float* __restrict__ weights, int8_t* __restrict__ xq,
    float* __restrict__ xscale, int* __restrict__ clear, int n_clear, int blocks) {
  __shared__ __align__(16) float logits[kMoeMaxExperts];
  __shared__ uint32_t keys[kMoeMaxExperts];
  __shared__ int chosen[kMoeMaxTopK];
  __shared__ float dots[kMoeMaxExperts / 2];  // [expert of the block][part]; 2 blocks at least
  __shared__ unsigned tops[kRouteWarps];
  grid_dependency_wait();  // the call before may still use the workspace, x may not be there yet
  allow_dependent_launch();
  // the first block has to be there before the others write to it: they arrive here and wait
  // just before they do
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  constexpr int kBatch = kXBf16 && kRBf16 ? 8 : 4;  // vectors in flight per lane
  const int t = blockIdx.x / blocks, part = blockIdx.x % blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = blockIdx.x * kRouteThreads + threadIdx.x; i < n_clear; i += gridDim.x * kRouteThreads) clear[i] = 0;
  const char* xr = static_cast<const char*>(x) + row_offset(t, D, kXBf16);
  // `share` warps (a power of two) to an expert, experts part, part + blocks, ... of the token
  const int experts = max(1, (E - part + blocks - 1) / blocks);  // one that is not there at least
  int share = 1;
  while (2 * share * ((E + 7) / 8) <= kRouteWarps) share *= 2;
  // of the block's experts this warp has number group, group + groups, ...: `mine` of them
  const int group = warp / share, groups = kRouteWarps / share, mine = (experts - group + groups - 1) / groups;
  const int stride = 32 * share, first = (warp % share) * 32 + lane;  // of the lane's vectors
  const int steps = (D / 8 + stride - 1) / stride;
  unsigned m = 0u;  // bits of the largest |x|; those of a NaN are larger still
  // `kExperts` of the warp's experts at once, `kSteps` vectors of each in flight
  auto products = [&](auto n_experts, auto n_steps) {
    constexpr int kExperts = decltype(n_experts)::value, kSteps = decltype(n_steps)::value;
    for (int i0 = 0; i0 < mine; i0 += kExperts) {
      const char* rr[kExperts];  // behind the last expert: the last again
      float s[kExperts];
#pragma unroll
      for (int i = 0; i < kExperts; ++i) {
        const int e = min(part + blocks * (group + groups * min(i0 + i, mine - 1)), E - 1);
        rr[i] = static_cast<const char*>(router) + row_offset(e, D, kRBf16);
        s[i] = 0.0f;
      }
      for (int k = 0; k < steps; k += kSteps) {
        Raw8<kXBf16> a[kSteps];
        Raw8<kRBf16> b[kSteps][kExperts];
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          const int c = min(first + stride * (k + u), D / 8 - 1);
          a[u] = load_raw8<kXBf16, true>(xr, c);  // kept in this order: all before the first use
#pragma unroll
          for (int i = 0; i < kExperts; ++i) b[u][i] = load_raw8<kRBf16, true>(rr[i], c);
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
          float x8[8];
          unpack8<kXBf16>(a[u], x8);
#pragma unroll
          for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x8[j]) & 0x7fffffffu);
          const bool in = first + stride * (k + u) < D / 8;
#pragma unroll
          for (int i = 0; i < kExperts; ++i) {
            float r8[8];
            unpack8<kRBf16>(b[u][i], r8);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[i] = fmaf(x8[j], in ? r8[j] : 0.0f, s[i]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kExperts; ++i) {
        s[i] = warp_sum(s[i]);
        if (lane == 0 && i0 + i < mine) dots[(group + groups * (i0 + i)) * share + warp % share] = s[i];
      }
    }
  };
  if (mine == 1)
    products(std::integral_constant<int, 1>{}, std::integral_constant<int, kBatch>{});
  else  // a row's vectors serve four experts (64 tokens, 512 experts of 4096: 128 -> 111 us, whole layer)
    products(std::integral_constant<int, 4>{}, std::integral_constant<int, kBatch / 4>{});
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) tops[warp] = m;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (threadIdx.x < experts && part + blocks * static_cast<int>(threadIdx.x) < E) {
    float logit = 0.0f;
    for (int j = 0; j < share; ++j) logit += dots[threadIdx.x * share + j];
    st_cluster_f32(smem_u32(logits + part + blocks * threadIdx.x), 0, logit);
  }
  const float a = __uint_as_float(__reduce_max_sync(0xffffffffu, tops[lane % kRouteWarps]));
  const bool fine = a <= kFloatMax;
  if (!fine && threadIdx.x == 0) record_status(kStatusNonfinite);
  const float f = fine && a > 0.0f ? __fdiv_rn(127.0f, a) : 0.0f;
  for (int c = part * kRouteThreads + threadIdx.x; c < D / 8; c += blocks * kRouteThreads) {
    float v[8];
    load8<kXBf16>(xr, c, v);
    uint32_t q[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i >> 2] |= (static_cast<uint32_t>(quant_i8(v[i], f)) & 0xffu) << (8 * (i & 3));
    reinterpret_cast<uint2*>(xq + static_cast<size_t>(t) * D)[c] = make_uint2(q[0], q[1]);
  }
  cluster_barrier();  // every block's logits are in the first one's shared memory
  if (part != 0) return;
  if (threadIdx.x == 0) xscale[t] = fine ? __fdiv_rn(a, 127.0f) : 0.0f;
  moe_top_k<kRouteThreads>(logits, E, top_k, renorm, keys, chosen, ids + t * top_k, weights + t * top_k);
}

// ------------------------------------------------------------------------------- experts
constexpr int kMoeThreads = 256;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeRingBytes = 8 * 1024;    // weights a warp keeps in flight
constexpr int kMoeSumBytes = 32 * 1024;    // integer sums of a run

// The pairs by expert: block-wide, in shared memory.
struct MoeGroups {
  int active;                       // experts with a pair
  int expert[kMoeMaxExperts];       // their indexes, ascending
  int begin[kMoeMaxExperts + 1];    // their pairs are list[begin[a] .. begin[a + 1])
  int work[kMoeMaxExperts + 1];     // turns over a tile (one per group of columns), added up
  short list[kMoeMaxTokens * kMoeMaxTopK];
  int cursor[kMoeMaxExperts];
};

// cols pairs make a group; an expert has `per` tiles.
__device__ __forceinline__ void moe_group(MoeGroups& g, const int* ids, int pairs, int E, int cols,
                                          int per) {
  constexpr int kPer = kMoeMaxTokens * kMoeMaxTopK / kMoeThreads;
  int mine[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int p = i * kMoeThreads + threadIdx.x;
    mine[i] = p < pairs ? __ldcg(ids + p) : -1;
  }
  for (int e = threadIdx.x; e < E; e += kMoeThreads) g.cursor[e] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (mine[i] >= 0) atomicAdd(&g.cursor[mine[i]], 1);
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int a0 = 0, p0 = 0, w0 = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane, n = e < E ? g.cursor[e] : 0, turns = (n + cols - 1) / cols;
      const uint32_t has = __ballot_sync(0xffffffffu, n > 0);
      int before = (turns << 16) | n;  // of the lanes up to this one (at most 1024 pairs in all)
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
      }
      if (n > 0) {
        const int a = a0 + __popc(has & ((1u << lane) - 1u));
        g.expert[a] = e;
        g.begin[a] = p0 + (before & 0xffff) - n;
        g.cursor[e] = g.begin[a];
        g.work[a] = (w0 + (before >> 16) - turns) * per;
      }
      a0 += __popc(has);
      const int all = __shfl_sync(0xffffffffu, before, 31);
      p0 += all & 0xffff;
      w0 += all >> 16;
    }
    if (lane == 0) {
      g.active = a0;
      g.begin[a0] = p0;
      g.work[a0] = w0 * per;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (mine[i] >= 0)
      g.list[atomicAdd(&g.cursor[mine[i]], 1)] = static_cast<short>(i * kMoeThreads + threadIdx.x);
  __syncthreads();
}

// Everything that the two expert kernels read and write.
struct MoeArgs {
  const int* ids;         // [pairs]
  const int8_t* xq;       // [M][D]
  const float* xscale;    // [M]
  const uint8_t *gate, *up, *down;
  const float *gate_gamma, *up_gamma, *down_gamma;
  float* inner;           // [pairs][F]
  unsigned* amax;         // [pairs] bits of the largest |inner|; starts at 0
  const int8_t* hq;       // [pairs][F] codes of inner
  const float* hscale;    // [pairs]
  float* part;            // [pairs][D] the experts' outputs
  int M, E, D, F, top_k, act;
  int wk, passes;         // warps of a block along K, and turns of all of them
};

// A run: up to kRunTiles tiles of one expert, for one group of 8 NT of its pairs.
struct MoeRun {
  int a, tile, tiles, group, groups;
};

// The 16-row tiles of the active experts, in order, are dealt out in equal stretches to the blocks,
// two per SM (one's barriers and loads of codes hide behind the other's stream). Within a
// block wk warps split K and the others take further tiles. As in few_tokens_kernel a warp
// holds its part of the codes in registers, streams its weights through a ring of its own that
// runs ahead across tiles and runs, and adds its sums to the block's; a run ends with a
// barrier, where they become what kDown says below. Bound by the weights' bytes up to 8 tokens
// per expert (16 tokens of 64 experts: the gate and up stream takes 46 of 53 thousand cycles
// that its bytes need, beside 20 for loading codes, joins and the first and last tiles), by
// instructions beyond (a turn of 16 columns costs 170 instructions per KB of weights). Codes in
// shared memory instead, with warps that take whole rows, measured the same at 64 tokens and
// slower below (16 tokens of 64 experts: 72 against 82 us).
//   kDown = false: inner = act(G) U of the run's rows and pairs, and their maximum;
//   kDown = true:  the experts' outputs.
template <int NT, int S, int MODE, bool kDown>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_expert_kernel(const MoeArgs p) {
  constexpr int kMats = kDown ? 1 : 2;
  constexpr int kAhead = kMoeRingBytes / 1024 / S;
  constexpr int kCols = 8 * NT;
  constexpr int kRunTiles = kMoeSumBytes / (kMats * 16 * kCols * 4);
  extern __shared__ __align__(16) uint8_t ring_all[];  // then the sums [matrix][row of the run][column]
  int* sums = reinterpret_cast<int*>(ring_all + kMoeWarps * kMoeRingBytes);
  __shared__ MoeGroups groups;
  __shared__ unsigned top[kCols];
  __shared__ float factor[kMats][kCols];  // scale of a pair's codes times gamma
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int N = kDown ? p.D : p.F, K = kDown ? p.F : p.D, pairs = p.M * p.top_k;
  const int chunks = K / 64, per = N / 16;  // tiles of an expert (N % 64 == 0)
  const int wr = warp / p.wk, WR = kMoeWarps / p.wk, wk = warp % p.wk;
  const size_t pitch = static_cast<size_t>(K / 4), matrix = static_cast<size_t>(N) * pitch;
  for (int i = threadIdx.x; i < kMoeSumBytes / 16; i += kMoeThreads)
    reinterpret_cast<uint4*>(sums)[i] = make_uint4(0u, 0u, 0u, 0u);
  // The pairs were chosen by the kernel before the gate and up products, which let this one
  // start only after it had waited for that: the down kernel may read them at once.
  if (!kDown) grid_dependency_wait();
  moe_group(groups, p.ids, pairs, p.E, kCols, per);
  if (!kDown) allow_dependent_launch();
  // The block's stretch: from the first tile at or behind its share of the work to that of the
  // next block, as (expert, tile).
  auto share = [&](int block, int& a, int& tile) {
    const int at = static_cast<int>(static_cast<long long>(groups.work[groups.active]) * block / gridDim.x);
    int lo = 0, hi = groups.active;  // the last a with work[a] <= at
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (groups.work[mid] <= at) lo = mid; else hi = mid;
    }
    const int turns = (groups.work[lo + 1] - groups.work[lo]) / per;
    a = lo;
    tile = (at - groups.work[lo] + turns - 1) / turns;
    if (tile == per) {
      ++a;
      tile = 0;
    }
  };
  int end_a, end_tile;
  share(blockIdx.x + 1, end_a, end_tile);
  auto open = [&](const MoeRun& r) { return r.a < end_a || (r.a == end_a && r.tile < end_tile); };
  auto start = [&](MoeRun& r) {  // the run that begins at (r.a, r.tile)
    if (r.tile >= per) {
      ++r.a;
      r.tile = 0;
    }
    if (!open(r)) return;
    r.tiles = min((r.a == end_a ? end_tile : per) - r.tile, kRunTiles);
    r.group = 0;
    r.groups = (groups.work[r.a + 1] - groups.work[r.a]) / per;
  };
  auto next = [&](MoeRun& r) {
    if (++r.group < r.groups) return;
    r.tile += r.tiles;
    start(r);
  };
  // ---- the stream: units (run, turn, tile, matrix) in the order in which they are used
  MoeRun fr;
  int f_turn = 0, f_tile = wr, f_mat = 0;
  share(blockIdx.x, fr.a, fr.tile);
  start(fr);
  MoeRun run = fr;
  const uint32_t ring = smem_u32(ring_all) + warp * kMoeRingBytes + lane * 16;
  const ptrdiff_t other = kDown ? 0 : p.up - p.gate;  // from a tile of gate to that of up
  const uint8_t* f_ptr = nullptr;  // this lane's row of the tile to fetch (of gate or down)
  int f_chunk = 0;
  auto seek = [&]() {
    while (open(fr) && f_tile >= fr.tiles) {  // runs with fewer tiles than warps
      f_tile = wr;
      if (++f_turn >= p.passes) {
        f_turn = 0;
        next(fr);
      }
    }
    f_ptr = nullptr;
    if (!open(fr)) return;
    f_chunk = 4 * S * (f_turn * p.wk + wk) + t4;
    f_ptr = (kDown ? p.down : p.gate) + groups.expert[fr.a] * matrix + ((fr.tile + f_tile) * 16 + g) * pitch;
  };
  auto fetch = [&](uint32_t slot) {
    if (f_ptr) {
      const uint8_t* a = f_mat ? f_ptr + other : f_ptr;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int at = 16 * min(f_chunk + 4 * s, chunks - 1);
        cp_async16(slot + s * 1024, a + at);
        cp_async16(slot + s * 1024 + 512, a + 8 * pitch + at);
      }
      if (++f_mat == kMats) {
        f_mat = 0;
        f_tile += WR;
        if (f_tile < fr.tiles) f_ptr += 16 * WR * pitch; else seek();
      }
    }
    cp_async_commit();
  };
  seek();
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) fetch(ring + i * S * 1024);
  if (kDown) grid_dependency_wait();
  // ---- the runs
  uint4 q[S][NT][4];
  int minus[NT][2];
  int held_a = -1, held_group = -1;
  uint32_t slot = ring;
  while (open(run)) {
    const int e = groups.expert[run.a], first = groups.begin[run.a] + run.group * kCols;
    const int n = min(groups.begin[run.a + 1] - first, kCols);  // pairs of the group
    if (threadIdx.x < n) {  // read behind the barrier that ends the run's products
      const int pair = groups.list[first + threadIdx.x];
      if (kDown) {
        factor[0][threadIdx.x] = __fmul_rn(p.hscale[pair], p.down_gamma[e]);
      } else {
        const float s = p.xscale[pair / p.top_k];
        factor[0][threadIdx.x] = __fmul_rn(s, p.gate_gamma[e]);
        factor[kMats - 1][threadIdx.x] = __fmul_rn(s, p.up_gamma[e]);
        top[threadIdx.x] = 0u;
      }
    }
    for (int turn = 0; turn < p.passes; ++turn) {
      if (p.passes > 1 || held_a != run.a || held_group != run.group) {
        held_a = run.a;
        held_group = run.group;
        const int c = 4 * S * (turn * p.wk + wk) + t4;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int col = MODE == kPairs ? g >> 1 : 8 * j + g;
          const bool here = col < n;
          const int pair = here ? groups.list[first + col] : 0;
          int sum = 0;
          const uint4* row = reinterpret_cast<const uint4*>(
              (kDown ? p.hq : p.xq) + static_cast<size_t>(kDown ? pair : pair / p.top_k) * K);
#pragma unroll
          for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = (here && c + 4 * s < chunks) ? row[4 * (c + 4 * s) + i]
                                                           : make_uint4(0u, 0u, 0u, 0u);
              sum = dot_ones(v, sum);
              q[s][j][i] = MODE == kPairs && (g & 1) ? next_plane(v) : v;
            }
          minus_of<MODE>(sum, minus[j]);
        }
      }
      for (int i = wr; i < run.tiles; i += WR)
#pragma unroll 1
        for (int m = 0; m < kMats; ++m) {
          int acc[planes(MODE)][NT][4];
          ternary_clear<NT, MODE>(acc, minus);
          cp_async_wait<kAhead - 1>();
#pragma unroll
          for (int s = 0; s < S; ++s) {
            const uint4 wa = ld_shared_v4(slot + s * 1024), wb = ld_shared_v4(slot + s * 1024 + 512);
            ternary_step<NT, MODE>(acc, wa, wb, q[s]);
          }
          fetch(slot);
          slot = slot + S * 1024 == ring + kAhead * S * 1024 ? ring : slot + S * 1024;
          ternary_add<NT, MODE>(acc, sums + (m * kRunTiles + i) * 16 * kCols, n);
        }
    }
    __syncthreads();
    // ---- the join: 16 threads take the rows of a tile for one pair
    for (int u = threadIdx.x >> 4; u < run.tiles * n; u += kMoeThreads / 16) {
      const int r = threadIdx.x & 15, i = u / n, col = u - i * n;
      const int pair = groups.list[first + col], row = (run.tile + i) * 16 + r;
      int* from = sums + (i * 16 + r) * kCols + col;
      if (kDown) {
        p.part[static_cast<size_t>(pair) * N + row] = __fmul_rn(__int2float_rn(*from), factor[0][col]);
      } else {
        int* from_up = from + kRunTiles * 16 * kCols;
        const float G = __fmul_rn(__int2float_rn(*from), factor[0][col]);
        const float U = __fmul_rn(__int2float_rn(*from_up), factor[kMats - 1][col]);
        const float v = __fmul_rn(moe_act(G, p.act), U);
        *from_up = 0;
        p.inner[static_cast<size_t>(pair) * N + row] = v;
        unsigned most = __float_as_uint(fabsf(v));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffu << (lane & 16), most, o));
        if (r == 0) atomicMax(&top[col], most);
      }
      *from = 0;
    }
    __syncthreads();
    if (!kDown) {
      if (threadIdx.x < n) atomicMax(p.amax + groups.list[first + threadIdx.x], top[threadIdx.x]);
      __syncwarp();  // top and factor are written again by the same threads
    }
    next(run);
  }
}

// y_t = sum_s w[t,s] part[t top_k + s], in the order of the slots.
template <bool kOBf16>
__global__ void __launch_bounds__(256) moe_combine_kernel(const float* __restrict__ part,
                                                         const float* __restrict__ weights, int D,
                                                         int top_k, void* __restrict__ y) {
  grid_dependency_wait();
  const int t = blockIdx.y, d = blockIdx.x * 256 + threadIdx.x;
  if (d >= D) return;
  float s = 0.0f;
#pragma unroll 4
  for (int k = 0; k < top_k; ++k)
    s = fmaf(weights[t * top_k + k], part[static_cast<size_t>(t * top_k + k) * D + d], s);
  const size_t at = static_cast<size_t>(t) * D + d;
  if (kOBf16) static_cast<__nv_bfloat16*>(y)[at] = __float2bfloat16_rn(s);
  else static_cast<float*>(y)[at] = s;
}

}  // namespace bl
