// sf_lora_add: low-rank adapters of many requests beside a shared projection,
//   out[t] = y[t] + scale_a B_a (A_a x[t]),  a the adapter of row t.
//
// A thread-block cluster takes a window of rows and the window's distinct
// adapters, one after another (with few windows, several clusters share the
// adapters of one).  For an adapter it lists the rows that use it, whatever
// their order, and works on 16 of them at a time, in one launch:
//  * h = x A^T: the cluster's blocks split K, a block's warps split its part
//    again (mma.m16n8k16 bf16, fragments straight from global memory: the k
//    order inside a product is free, so lane t of a row's four takes 16
//    contiguous bytes).  Warps add up in shared memory, blocks through
//    distributed shared memory, both in a fixed order;
//  * out = y + h B^T: the blocks split N.  h enters as three bf16 terms (24
//    bits), so the second product keeps fp32 accuracy: h is fp32, and its
//    rounding to bf16 would show in the fp32 output.
// What the second product reads does not wait for the first: a warp's first B
// is loaded, and y prefetched to L2, before h is summed.  Bound by latency for
// a decode batch (a chain of two weight reads and a cluster barrier), by the
// reads and writes of y and out for prompts.
#include <algorithm>

#include <cooperative_groups.h>

#include "sf_internal.h"

namespace {

namespace cg = cooperative_groups;

constexpr int kLoraMaxRank = 128;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWindow = 64;
constexpr int kRows = 16;  // rows worked on at a time
constexpr int kNB = 4;     // tiles of 8 outputs that a warp takes at a time

__device__ __forceinline__ void bmma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct LoraArgs {
  sf_lora_args a;
  int window;  // rows of a window
  int share;   // clusters per window
  int log_blocks;
  int vec;  // rows of y and out allow 8-byte accesses
};

// KS: steps of 16 ranks that the second product takes (rank <= 16 KS, zeros beyond it).
template <int KS>
struct Shape {
  static constexpr int RK = 16 * KS;
  static constexpr int RB = RK < 64 ? RK : 64;  // rank columns of one pass over x
  static constexpr int KB = KS < 4 ? KS : 4;    // k steps whose B a warp holds
  static constexpr int PITCH = RK + 8;
};

// The block's shared memory.
template <int KS>
struct Shared {
  float part[kWarps][kRows][Shape<KS>::RB + 1];   // the warps' sums of one pass
  float h[kRows * Shape<KS>::RK];                 // the block's sums
  uint16_t term[3][kRows][Shape<KS>::PITCH];      // the cluster's sums times the scale, as bf16 terms
  int ids[kMaxWindow], list[kMaxWindow], bare[kMaxWindow];
  int list_n, bare_n;
  unsigned leads[2];  // rows that are the first of their adapter
};

// Lists the window's rows with this id; a warp's work.
__device__ __forceinline__ void list_rows(const int* ids, int id, int rows, int* list, int* count) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int q = 0; q < rows; q += 32) {
    const unsigned m = __ballot_sync(0xffffffffu, q + lane < rows && ids[q + lane] == id);
    if (m >> lane & 1) list[n + __popc(m & ((1u << lane) - 1))] = q + lane;
    n += __popc(m);
  }
  if (lane == 0) *count = n;
}

// Rows list[0 .. n) (n <= 16) of adapter id.  Every block of the cluster calls it with the same arguments.  `again`:
// the blocks' sums of an earlier call may still be read.
template <int KS>
__device__ void lora_rows(const LoraArgs& P, Shared<KS>& S, const int* list, int n, int row0, int id, bool again,
                          cg::cluster_group& cluster) {
  using C = Shape<KS>;
  const sf_lora_args& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int blocks = 1 << P.log_blocks, block = static_cast<int>(cluster.block_rank());
  const float scale = a.scale[id];

  // this block's run of 8-column output tiles
  const uint32_t tiles = (a.N + 7u) / 8u;
  const int t0 = static_cast<int>(static_cast<uint64_t>(tiles) * block >> P.log_blocks);
  const int t1 = static_cast<int>(static_cast<uint64_t>(tiles) * (block + 1) >> P.log_blocks);
  const int r[2] = {g, g + 8};
  const uint16_t* x[2];
  const float* y[2];
  float* out[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const int64_t row = row0 + list[r[z] < n ? r[z] : 0];
    x[z] = a.x + row * a.x_stride + 8 * t;
    y[z] = a.y ? a.y + row * a.y_stride + 2 * t : nullptr;
    out[z] = a.out + row * a.out_stride + 2 * t;
  }
  const uint16_t* const Bw = a.B + (static_cast<int64_t>(id) * a.N + g) * a.rank + 4 * t;
  uint2 b[C::KB][kNB];
  auto load_b = [&](int tile, int q0) {
    const uint16_t* from = Bw + static_cast<int64_t>(8 * tile) * a.rank + 16 * q0;
    const int cols = min(t1 - tile, kNB);  // tiles there are
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const bool in = j < cols && 8 * (tile + j) + g < a.N;
#pragma unroll
      for (int q = 0; q < C::KB; ++q)
        b[q][j] = in && 16 * (q0 + q) + 4 * t < a.rank
                      ? *reinterpret_cast<const uint2*>(from + (8 * j) * a.rank + 16 * q)
                      : make_uint2(0, 0);
    }
  };
  load_b(t0 + warp * kNB, 0);
  if (a.y) {  // y's lines of this block, spread over the warps
    const int c0 = 8 * t0, c1 = min(8 * t1, a.N);
    for (int q = warp; q < n; q += kWarps)
      for (int c = c0 + 32 * lane; c < c1; c += 1024)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.y + static_cast<int64_t>(row0 + list[q]) * a.y_stride + c));
  }

  // h: this warp's run of 64-channel steps
  const uint32_t steps = (a.K + 63u) / 64u, w = block * kWarps + warp;
  const int s0 = static_cast<int>(static_cast<uint64_t>(steps) * w >> (P.log_blocks + 3));
  const int s1 = static_cast<int>(static_cast<uint64_t>(steps) * (w + 1) >> (P.log_blocks + 3));
  const uint16_t* const Aw = a.A + (static_cast<int64_t>(id) * a.rank + g) * a.K + 8 * t;
#pragma unroll
  for (int p = 0; p < C::RK / C::RB; ++p) {
    const int r0 = p * C::RB;
    if (p > 0 && r0 >= a.rank) break;
    float acc[C::RB / 8][4] = {};
#pragma unroll 2
    for (int k = 64 * s0; k < 64 * s1; k += 32) {
      const bool in = k + 8 * t < a.K;
      uint4 xv[2], av[C::RB / 8];
#pragma unroll
      for (int j = 0; j < C::RB / 8; ++j)
        av[j] = in && r0 + 8 * j < a.rank
                    ? *reinterpret_cast<const uint4*>(Aw + static_cast<int64_t>(r0 + 8 * j) * a.K + k)
                    : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int z = 0; z < 2; ++z)
        xv[z] = in && r[z] < n ? *reinterpret_cast<const uint4*>(x[z] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < C::RB / 8; ++j) {
        bmma(acc[j], xv[0].x, xv[1].x, xv[0].y, xv[1].y, av[j].x, av[j].y);
        bmma(acc[j], xv[0].z, xv[1].z, xv[0].w, xv[1].w, av[j].z, av[j].w);
      }
    }
    if (p > 0) __syncthreads();  // the sums of the pass before are read
#pragma unroll
    for (int j = 0; j < C::RB / 8; ++j)
#pragma unroll
      for (int z = 0; z < 4; ++z) S.part[warp][g + 8 * (z >> 1)][8 * j + 2 * t + (z & 1)] = acc[j][z];
    __syncthreads();
    if (p == 0 && again) cluster.barrier_wait();  // the other blocks have read this one's sums of the call before
    for (int e = tid; e < kRows * C::RB; e += kThreads) {
      const int row = e / C::RB, c = e % C::RB;
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += S.part[v][row][c];
      S.h[row * C::RK + r0 + c] = sum;
    }
    if (p + 1 < C::RK / C::RB && r0 + C::RB >= a.rank)  // ranks of the next pass that there are not
      for (int e = tid; e < kRows * C::RB; e += kThreads) S.h[e / C::RB * C::RK + r0 + C::RB + e % C::RB] = 0.f;
  }
  cluster.sync();
  for (int e = tid; e < kRows * C::RK; e += kThreads) {
    float v[8], sum = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = c < blocks ? cluster.map_shared_rank(S.h, c)[e] : 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) sum += v[c];
    sum *= scale;
#pragma unroll
    for (int z = 0; z < 3; ++z) {
      const __nv_bfloat16 t16 = __float2bfloat16_rn(sum);
      S.term[z][e / C::RK][e % C::RK] = __bfloat16_as_ushort(t16);
      sum -= __bfloat162float(t16);
    }
  }
  cluster.barrier_arrive();
  __syncthreads();

  for (int tile = t0 + warp * kNB; tile < t1; tile += kWarps * kNB) {
    const bool full = P.vec && tile + kNB <= t1 && 8 * (tile + kNB) <= a.N;
    float2 v[2][kNB] = {};
    if (a.y) {
#pragma unroll
      for (int z = 0; z < 2; ++z)
        if (r[z] < n) {
          const float* from = y[z] + 8 * tile;
          if (full) {
#pragma unroll
            for (int j = 0; j < kNB; ++j) v[z][j] = *reinterpret_cast<const float2*>(from + 8 * j);
          } else {
#pragma unroll
            for (int j = 0; j < kNB; ++j) {
              if (tile + j >= t1) continue;
              if (8 * (tile + j) + 2 * t < a.N) v[z][j].x = from[8 * j];
              if (8 * (tile + j) + 2 * t + 1 < a.N) v[z][j].y = from[8 * j + 1];
            }
          }
        }
    }
    float d[kNB][4] = {};
#pragma unroll
    for (int q0 = 0; q0 < KS; q0 += C::KB) {
#pragma unroll
      for (int q = 0; q < C::KB; ++q)
#pragma unroll
        for (int z = 2; z >= 0; --z) {  // the small terms first
          const uint16_t* from = &S.term[z][g][16 * (q0 + q) + 4 * t];
          const uint2 lo = *reinterpret_cast<const uint2*>(from);
          const uint2 hi = *reinterpret_cast<const uint2*>(from + 8 * C::PITCH);
#pragma unroll
          for (int j = 0; j < kNB; ++j) bmma(d[j], lo.x, hi.x, lo.y, hi.y, b[q][j].x, b[q][j].y);
        }
      if (q0 + C::KB < KS)
        load_b(tile, q0 + C::KB);
      else if (tile + kWarps * kNB < t1)
        load_b(tile + kWarps * kNB, 0);
    }
#pragma unroll
    for (int z = 0; z < 2; ++z)
      if (r[z] < n) {
        float* to = out[z] + 8 * tile;
#pragma unroll
        for (int j = 0; j < kNB; ++j) {
          const float2 s = make_float2(v[z][j].x + d[j][2 * z], v[z][j].y + d[j][2 * z + 1]);
          if (full) {
            *reinterpret_cast<float2*>(to + 8 * j) = s;
          } else if (tile + j < t1) {
            if (8 * (tile + j) + 2 * t < a.N) to[8 * j] = s.x;
            if (8 * (tile + j) + 2 * t + 1 < a.N) to[8 * j + 1] = s.y;
          }
        }
      }
  }
}

template <int KS>
__global__ void __launch_bounds__(kThreads, 2) lora_kernel(const __grid_constant__ LoraArgs P) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<KS>& S = *reinterpret_cast<Shared<KS>*>(smem);
  const sf_lora_args& a = P.a;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, block = static_cast<int>(cluster.block_rank());
  const int task = blockIdx.x >> P.log_blocks, window = task / P.share, turn = task % P.share;
  const int row0 = window * P.window, rows = min(P.window, a.T - row0);
  if (tid < kMaxWindow) {
    int id = -1;
    if (tid < rows) {
      int at = row0 + tid;
      if (a.row_of) at = a.row_of[at];
      if (at >= 0 && at < a.n_ids) id = a.ids[at];
      if (id < 0 || id >= a.n_adapters) id = -1;
    }
    S.ids[tid] = id;
  }
  __syncthreads();
  if (tid < kMaxWindow) {
    bool first = S.ids[tid] >= 0;
    for (int q = 0; q < tid; ++q) first &= S.ids[q] != S.ids[tid];
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if ((tid & 31) == 0) S.leads[tid >> 5] = m;
  } else if (tid < kMaxWindow + 32) {
    list_rows(S.ids, -1, rows, S.bare, &S.bare_n);
  }
  __syncthreads();

  // The window's adapters in the order of their first rows; this cluster takes every share-th.
  unsigned long long lead = S.leads[0] | static_cast<unsigned long long>(S.leads[1]) << 32;
  bool again = false;
  for (int seen = 0; lead != 0; lead &= lead - 1, ++seen) {
    if (seen % P.share != turn) continue;
    const int id = S.ids[__ffsll(lead) - 1];
    __syncthreads();  // the list before is done with
    if (tid < 32) list_rows(S.ids, id, rows, S.list, &S.list_n);
    __syncthreads();
    const int n = S.list_n;
    for (int k = 0; k < n; k += kRows) {
      lora_rows<KS>(P, S, S.list + k, min(kRows, n - k), row0, id, again, cluster);
      again = true;
    }
  }

  // Rows without an adapter, spread over the window's clusters, four at a time.
  if (a.out != a.y) {
    const int c0 = static_cast<int>(static_cast<int64_t>(a.N) * block >> P.log_blocks);
    const int c1 = static_cast<int>(static_cast<int64_t>(a.N) * (block + 1) >> P.log_blocks);
    for (int q = 4 * turn; q < S.bare_n; q += 4 * P.share)
      for (int c = c0 + tid; c < c1; c += kThreads) {
        float v[4] = {};
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (a.y && q + k < S.bare_n) v[k] = a.y[static_cast<int64_t>(row0 + S.bare[q + k]) * a.y_stride + c];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (q + k < S.bare_n) a.out[static_cast<int64_t>(row0 + S.bare[q + k]) * a.out_stride + c] = v[k];
      }
  }
  if (again) cluster.barrier_wait();  // the other blocks have read this one's sums
}

template <int KS>
sf_status launch(const LoraArgs& P, int clusters, cudaStream_t s) {
  const size_t smem = sizeof(Shared<KS>);
  if (smem > 48 * 1024)
    SF_CHECK_CUDA(
        cudaFuncSetAttribute(lora_kernel<KS>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(clusters << P.log_blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 1 << P.log_blocks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  SF_CHECK_CUDA(cudaLaunchKernelEx(&cfg, lora_kernel<KS>, P));
  return sf::check_launch("lora_kernel");
}

}  // namespace

extern "C" sf_status sf_lora_add(const sf_lora_args* a, sf_stream_t stream) {
  const char* what = "sf_lora_add";
  SF_REQUIRE(a, "%s: null arguments", what);
  SF_REQUIRE(a->T >= 0 && a->n_ids >= 0, "%s: need T >= 0 and n_ids >= 0", what);
  SF_REQUIRE(a->n_adapters >= 1 && a->N >= 1, "%s: need n_adapters >= 1 and N >= 1", what);
  SF_REQUIRE(a->K >= 8 && a->K % 8 == 0, "%s: K must be a positive multiple of 8", what);
  SF_REQUIRE(a->rank >= 8 && a->rank <= kLoraMaxRank && a->rank % 8 == 0,
             "%s: rank must be a multiple of 8 in [8, %d]", what, kLoraMaxRank);
  if (a->T == 0) return SF_OK;
  SF_REQUIRE(a->x && a->A && a->B && a->scale && a->out && (a->ids || a->n_ids == 0), "%s: null pointer", what);
  SF_REQUIRE(a->x_stride >= a->K && a->out_stride >= a->N && (!a->y || a->y_stride >= a->N),
             "%s: a row stride is below the row's length", what);
  SF_REQUIRE(sf::aligned(a->A, 16) && sf::aligned(a->B, 16) && sf::aligned(a->x, 16) && a->x_stride % 8 == 0,
             "%s: A, B and the rows of x must be 16-byte aligned", what);
  LoraArgs P{};
  P.a = *a;
  P.vec = a->N % 2 == 0 && sf::aligned(a->out, 8) && a->out_stride % 2 == 0 &&
          (!a->y || (sf::aligned(a->y, 8) && a->y_stride % 2 == 0));
  // Rows of one adapter are found within a window: wide windows for a decode batch, where the adapters' weights are
  // what is read, narrow ones for prompts, where more of them run at once.
  P.window = a->T <= 128 ? kMaxWindow : kRows;
  // Two blocks fit an SM.  Clusters of 8 share a window's adapters while there are few windows; with many windows a
  // cluster is as small as fills the SMs, so that fewer blocks wait for one another.
  const int windows = (a->T - 1) / P.window + 1, room = 2 * sf::sm_count();
  P.log_blocks = 3;
  while (P.log_blocks > 0 && static_cast<int64_t>(windows) << P.log_blocks > room) --P.log_blocks;
  P.share = std::max(1, std::min({P.window, a->T, a->n_adapters, (room >> P.log_blocks) / windows}));
  SF_REQUIRE(static_cast<int64_t>(windows) * P.share << P.log_blocks < (1ll << 31), "%s: T is too large", what);
  cudaStream_t s = sf::as_cuda(stream);
  const int clusters = windows * P.share;
  if (a->rank <= 16) return launch<1>(P, clusters, s);
  if (a->rank <= 32) return launch<2>(P, clusters, s);
  if (a->rank <= 64) return launch<4>(P, clusters, s);
  return launch<8>(P, clusters, s);
}
