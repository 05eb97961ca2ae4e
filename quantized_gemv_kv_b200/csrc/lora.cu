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
//    rounding to bf16 would show in the fp32 output.  Which column of a group of
//    32 a product's column stands for, and which rank a step's, is free too: so
//    that a lane's outputs and its ranks of a B row are 16 contiguous bytes (half
//    the memory instructions of the plain order; they were what bound it).
// What the second product reads does not wait for the first: a warp's first B
// is loaded, and y prefetched to L2, before h is summed.  Bound by latency for
// a decode batch (a chain of two weight reads and a cluster barrier), by the
// reads and writes of y and out for prompts.
#include <algorithm>

#include <cooperative_groups.h>

#include "launch.cuh"
#include "sf_internal.h"

namespace {

namespace cg = cooperative_groups;

constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxSize = 1 << 30;  // of K and N: the loops' indexes run past them by less than that
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxWindow = 64;
constexpr int kRows = 16;  // rows worked on at a time
constexpr int kNB = 4;     // tiles of 8 outputs that a warp takes at a time: a group of 32 columns

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
  int log_split;  // clusters that share an adapter's outputs, each with an h of its own
  int few;  // a decode batch
  int vec;  // rows of y and out allow 16-byte accesses
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

// Rows list[0 .. n) (n <= 16) of adapter id.  Every block of the cluster calls it with the same arguments.  run0: the
// first of the cluster's runs of outputs, one a block.  `again`: the blocks' sums of an earlier call may still be read.
template <int KS>
__device__ void lora_rows(const LoraArgs& P, Shared<KS>& S, const int* list, int n, int row0, int id, int run0,
                          bool again, cg::cluster_group& cluster) {
  using C = Shape<KS>;
  const sf_lora_args& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int blocks = 1 << P.log_blocks, block = static_cast<int>(cluster.block_rank());
  const float scale = a.scale[id];

  // this block's run of groups of 32 output columns
  const uint32_t groups = (a.N + 31u) / 32u;
  const uint32_t run = run0 + block;
  const int g0 = static_cast<int>(static_cast<uint64_t>(groups) * run >> (P.log_blocks + P.log_split));
  const int g1 = static_cast<int>(static_cast<uint64_t>(groups) * (run + 1) >> (P.log_blocks + P.log_split));
  const int r[2] = {g, g + 8};
  const uint16_t* x[2];
  const float* y[2];
  float* out[2];
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    const int64_t row = row0 + list[r[z] < n ? r[z] : 0];
    x[z] = a.x + row * a.x_stride + 8 * t;
    y[z] = a.y ? a.y + row * a.y_stride + 4 * t : nullptr;
    out[z] = a.out + row * a.out_stride + 4 * t;
  }
  // Column n of tile j is column 16 (j/2) + 4 (n/2) + 2 (j%2) + n%2 of the group, so that lane t's are 4 t .. 4 t + 3
  // and 16 more.  Rank i of step q is, for lane t's four, 32 (q/2) + 8 t + 4 (q%2) + i (rank <= 16: 4 t + i).
  const int bcol = 4 * (g >> 1) + (g & 1);
  const uint16_t* const Bw = a.B + (static_cast<int64_t>(id) * a.N + bcol) * a.rank + (KS == 1 ? 4 : 8) * t;
  uint2 b[C::KB][kNB];
  auto load_b = [&](int group, int q0) {
    const uint16_t* from = Bw + static_cast<int64_t>(32 * group) * a.rank + 16 * q0;
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const int c = 16 * (j >> 1) + 2 * (j & 1);
      const bool in = 32 * group + bcol + c < a.N;
      if constexpr (KS == 1) {
        b[0][j] = in && 4 * t < a.rank ? *reinterpret_cast<const uint2*>(from + c * a.rank) : make_uint2(0, 0);
      } else {
#pragma unroll
        for (int q = 0; q < C::KB; q += 2) {
          const uint4 v = in && 16 * (q0 + q) + 8 * t < a.rank
                              ? *reinterpret_cast<const uint4*>(from + c * a.rank + 16 * q)
                              : make_uint4(0, 0, 0, 0);
          b[q][j] = make_uint2(v.x, v.y);
          b[q + 1][j] = make_uint2(v.z, v.w);
        }
      }
    }
  };
  if (g0 + warp < g1) load_b(g0 + warp, 0);
  if (a.y) {  // y's lines of this block, spread over the warps
    const int c1 = min(32 * g1, a.N);
    for (int q = warp; q < n; q += kWarps)
      for (int c = 32 * (g0 + lane); c < c1; c += 1024)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.y + static_cast<int64_t>(row0 + list[q]) * a.y_stride + c));
  }

  // h: this warp's run of 64-channel steps
  const uint32_t steps = (a.K + 63u) / 64u, w = block * kWarps + warp;
  const int s0 = static_cast<int>(static_cast<uint64_t>(steps) * w >> (P.log_blocks + 3));
  const int s1 = static_cast<int>(static_cast<uint64_t>(steps) * (w + 1) >> (P.log_blocks + 3));
  const uint16_t* const Aw = a.A + (static_cast<int64_t>(id) * a.rank + g) * a.K + 8 * t;
#pragma unroll
  for (int p = 0; p < C::RK / C::RB; ++p) {  // (two passes only for ranks above 64)
    const int r0 = p * C::RB;
    float acc[C::RB / 8][4] = {};
    // A step's loads at once up to rank 32 (a decode batch's warp has one step: 8.6 us, 9.0 by halves); above, the
    // registers do not allow it (rank 64: 23.4 us, 21.8 by halves).
    constexpr int HALVES = KS <= 2 ? 2 : 1;
#pragma unroll 1
    for (int k = 64 * s0; k < 64 * s1; k += 32 * HALVES) {
      uint4 xv[HALVES][2], av[HALVES][C::RB / 8];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int at = k + 32 * h;
        const bool in = at + 8 * t < a.K;
#pragma unroll
        for (int j = 0; j < C::RB / 8; ++j)
          av[h][j] = in && r0 + 8 * j < a.rank
                         ? *reinterpret_cast<const uint4*>(Aw + static_cast<int64_t>(r0 + 8 * j) * a.K + at)
                         : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int z = 0; z < 2; ++z)
          xv[h][z] = in && r[z] < n ? *reinterpret_cast<const uint4*>(x[z] + at) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int j = 0; j < C::RB / 8; ++j) {
          bmma(acc[j], xv[h][0].x, xv[h][1].x, xv[h][0].y, xv[h][1].y, av[h][j].x, av[h][j].y);
          bmma(acc[j], xv[h][0].z, xv[h][1].z, xv[h][0].w, xv[h][1].w, av[h][j].z, av[h][j].w);
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
      S.h[row * C::RK + r0 + c] = r0 + c < a.rank ? sum : 0.f;  // (an infinite x times the zeros behind the rank)
    }
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
      __nv_bfloat16 t16 = __float2bfloat16_rn(sum);
      if (z == 0 && __hisinf(t16) && !isinf(sum)) t16 = __float2bfloat16_rz(sum);  // above bf16's largest: cut
      S.term[z][e / C::RK][e % C::RK] = __bfloat16_as_ushort(t16);
      sum = isinf(sum) ? 0.f : sum - __bfloat162float(t16);  // an infinity has no remainder
    }
  }
  cluster.barrier_arrive();
  __syncthreads();

  for (int group = g0 + warp; group < g1; group += kWarps) {
    const bool full = P.vec && 32 * (group + 1) <= a.N;
    const int left = a.N - 32 * group - 4 * t;  // columns from the lane's first on
    float v[2][2][4] = {};                      // rows x halves of the group
    if (a.y) {
#pragma unroll
      for (int z = 0; z < 2; ++z)
        if (r[z] < n) {
          const float* from = y[z] + 32 * group;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (full) {
              *reinterpret_cast<float4*>(v[z][h]) = *reinterpret_cast<const float4*>(from + 16 * h);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (16 * h + i < left) v[z][h][i] = from[16 * h + i];
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
          const uint16_t* from =
              &S.term[z][g][KS == 1 ? 4 * t : 16 * (q0 + (q & ~1)) + 8 * t + 4 * (q & 1)];
          const uint2 lo = *reinterpret_cast<const uint2*>(from);
          const uint2 hi = *reinterpret_cast<const uint2*>(from + 8 * C::PITCH);
#pragma unroll
          for (int j = 0; j < kNB; ++j) bmma(d[j], lo.x, hi.x, lo.y, hi.y, b[q][j].x, b[q][j].y);
        }
      if (q0 + C::KB < KS)
        load_b(group, q0 + C::KB);
      else if (group + kWarps < g1)
        load_b(group + kWarps, 0);
    }
#pragma unroll
    for (int z = 0; z < 2; ++z)
      if (r[z] < n) {
        float* to = out[z] + 32 * group;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = v[z][h][i] + d[2 * h + (i >> 1)][2 * z + (i & 1)];
          if (full) {
            *reinterpret_cast<float4*>(to + 16 * h) = make_float4(o[0], o[1], o[2], o[3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (16 * h + i < left) to[16 * h + i] = o[i];
          }
        }
      }
  }
}

template <int KS>
__global__ void __launch_bounds__(kThreads, 2) lora_kernel(const __grid_constant__ LoraArgs P) {
  sfd::wait_for_previous();
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<KS>& S = *reinterpret_cast<Shared<KS>*>(smem);
  const sf_lora_args& a = P.a;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, block = static_cast<int>(cluster.block_rank());
  const int cluster_id = blockIdx.x >> P.log_blocks, run0 = (cluster_id & ((1 << P.log_split) - 1)) << P.log_blocks;
  const int task = cluster_id >> P.log_split, window = task / P.share, turn = task % P.share;
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
      lora_rows<KS>(P, S, S.list + k, min(kRows, n - k), row0, id, run0, again, cluster);
      again = true;
    }
  }

  // Rows without an adapter, spread over the window's clusters: four columns, eight rows on their way at once.
  if (a.out != a.y && S.bare_n > turn) {
    const int64_t quads = (a.N + 3) / 4, run = run0 + block;
    const int p0 = static_cast<int>(quads * run >> (P.log_blocks + P.log_split));
    const int p1 = static_cast<int>(quads * (run + 1) >> (P.log_blocks + P.log_split));
    const int mine = (S.bare_n - 1 - turn) / P.share + 1;  // rows turn, turn + share, ...
    constexpr int kAhead = 8;
    for (int c = 4 * (p0 + tid); c < 4 * p1; c += 4 * kThreads)
      for (int q = 0; q < mine; q += kAhead) {
        const bool full = P.vec && c + 4 <= a.N;
        float v[kAhead][4] = {};
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (!a.y || q + k >= mine) continue;
          const float* from = a.y + static_cast<int64_t>(row0 + S.bare[turn + (q + k) * P.share]) * a.y_stride + c;
          if (full) {
            *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(from);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + i < a.N) v[k][i] = from[i];
          }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (q + k >= mine) continue;
          float* to = a.out + static_cast<int64_t>(row0 + S.bare[turn + (q + k) * P.share]) * a.out_stride + c;
          if (full) {
            *reinterpret_cast<float4*>(to) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + i < a.N) to[i] = v[k][i];
          }
        }
      }
  }
  if (again) cluster.barrier_wait();  // the other blocks have read this one's sums
}

template <int KS>
sf_status launch_lora(const LoraArgs& P, int clusters, cudaStream_t s) {
  const size_t smem = sizeof(Shared<KS>);
  static std::atomic<unsigned long long> told{0};
  const sf_status st = sf::allow_smem(lora_kernel<KS>, smem, told);
  if (st != SF_OK) return st;
  return sf::launch("lora_kernel", lora_kernel<KS>, dim3(clusters << P.log_blocks), kThreads, smem, 1 << P.log_blocks, s,
                    P);
}

}  // namespace

extern "C" sf_status sf_lora_add(const sf_lora_args* a, sf_stream_t stream) {
  const char* what = "sf_lora_add";
  SF_REQUIRE(a, "%s: null arguments", what);
  SF_REQUIRE(a->T >= 0 && a->n_ids >= 0, "%s: need T >= 0 and n_ids >= 0", what);
  SF_REQUIRE(a->n_adapters >= 1 && a->N >= 1 && a->N <= kLoraMaxSize, "%s: need n_adapters >= 1 and N >= 1, N <= 2^30",
             what);
  SF_REQUIRE(a->K >= 8 && a->K % 8 == 0 && a->K <= kLoraMaxSize, "%s: K must be a positive multiple of 8, at most 2^30",
             what);
  SF_REQUIRE(a->rank >= 8 && a->rank <= kLoraMaxRank && a->rank % 8 == 0,
             "%s: rank must be a multiple of 8 in [8, %d]", what, kLoraMaxRank);
  if (a->T == 0) return SF_OK;
  SF_REQUIRE(a->x && a->A && a->B && a->scale && a->out && (a->ids || a->n_ids == 0), "%s: null pointer", what);
  SF_REQUIRE(a->x_stride >= a->K && a->out_stride >= a->N && (!a->y || a->y_stride >= a->N),
             "%s: a row stride is below the row's length", what);
  SF_REQUIRE(a->out != a->y || a->out_stride == a->y_stride, "%s: out is y with another row stride", what);
  SF_REQUIRE(sf::aligned(a->A, 16) && sf::aligned(a->B, 16) && sf::aligned(a->x, 16) && a->x_stride % 8 == 0,
             "%s: A, B and the rows of x must be 16-byte aligned", what);
  LoraArgs P{};
  P.a = *a;
  P.vec = sf::aligned(a->out, 16) && a->out_stride % 4 == 0 && (!a->y || (sf::aligned(a->y, 16) && a->y_stride % 4 == 0));
  // Rows of one adapter are found within a window: wide windows for a decode batch, where the adapters' weights are
  // what is read, narrow ones for prompts, where more of them run at once.  Only the device knows which it is, so the
  // rule goes by T (us with windows of 64 / 32 / 16 rows: 256 rows of 16 adapters in any order 22 / 25 / 33; 512 in
  // runs of 100 rows 31 / 19 / 17).
  P.few = a->T <= 128;
  P.window = P.few ? kMaxWindow : a->T <= 512 ? 32 : kRows;
  // Two blocks fit an SM.  Clusters of 8 share a window's adapters while there are few windows; with many windows a
  // cluster is smaller, down to two rounds of blocks: while some sum h, others are at their outputs (2050 rows, rank
  // 32: 40 us; one round 44, four 48).  Prompts may hold many adapters a window all the same, and a cluster that has
  // none ends at once: four rounds more of them (36 us; eight, 42).
  const int windows = (a->T - 1) / P.window + 1, room = 2 * sf::sm_count();
  P.log_blocks = 3;
  while (P.log_blocks > 0 && static_cast<int64_t>(windows) << P.log_blocks > 2 * room) --P.log_blocks;
  const int most = ((a->T > 512 ? 4 * room : room) >> P.log_blocks) / windows;
  P.share = std::max(1, std::min({P.window, a->T, a->n_adapters, most}));
  // A wide projection's outputs are shared by two clusters while the SMs have room (64 rows, 16 adapters of rank 64, N =
  // 14336: 22 us; one cluster each takes 14% longer, clusters of 16 blocks instead 60%.  4 rows of rank 64, N = 4096 /
  // 2048 / 1024: 9.3 / 8.9 / 8.8 us shared, 10.6 / 9.3 / 8.9 not; but 16 rows of rank 16, N = 1024: 8.0 and 7.6, 64 rows
  // of rank 64, N = 1024: 12.8 and 12.3).
  P.log_split = P.few && a->N >= 2048 && static_cast<int64_t>(windows) * P.share * 2 << P.log_blocks <= room;
  SF_REQUIRE(static_cast<int64_t>(windows) * P.share << P.log_blocks < (1ll << 30), "%s: T is too large", what);
  cudaStream_t s = sf::as_cuda(stream);
  const int clusters = windows * P.share << P.log_split;
  if (a->rank <= 16) return launch_lora<1>(P, clusters, s);
  if (a->rank <= 32) return launch_lora<2>(P, clusters, s);
  if (a->rank <= 64) return launch_lora<4>(P, clusters, s);
  return launch_lora<8>(P, clusters, s);
}
