// sf_lora_add: low-rank adapters of many requests beside a shared projection,
//   out[t] = y[t] + scale_a B_a (A_a x[t]),  a the adapter of row t.
//
// A thread-block cluster takes a window of 64 rows and the window's distinct
// adapters, one after another (with few windows, several clusters share the
// adapters of one).  For an adapter it lists the rows that use it, whatever their
// order, and works on 16 or 32 of them at a time.  In one launch:
//  * h = x A^T: the cluster's blocks split K, a block's warps split its part
//    again (mma.m16n8k16 bf16, fragments straight from global memory: the k
//    order inside a product is free, so lane t of a row's four takes 16
//    contiguous bytes).  Warps add up in shared memory, blocks through
//    distributed shared memory, both in a fixed order;
//  * out = y + h B^T: the blocks split N.  h enters as three bf16 terms (24
//    bits), so the second product keeps fp32 accuracy: h is fp32, and its
//    rounding to bf16 would show in the fp32 output.
// Bound by latency for a decode batch (a chain of two weight reads and a
// cluster barrier), by the reads and writes of y and out for prompts.
#include <algorithm>

#include <cooperative_groups.h>

#include "sf_internal.h"

namespace {

namespace cg = cooperative_groups;

constexpr int kLoraMaxRank = 128;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kCluster = 8;
constexpr int kWindow = 64;
constexpr int kRB = 32;  // rank columns of one pass over x
constexpr int kNB = 4;   // tiles of 8 outputs that a warp takes at a time

__device__ __forceinline__ void bmma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct LoraArgs {
  sf_lora_args a;
  int rk;        // rank rounded up to 16
  int rows_cap;  // most rows that a block works on at a time: 16 or 32
  int share;     // clusters per window
  int vec;       // rows of y and out allow 8-byte accesses
};

// The block's shared memory.
struct Shared {
  float* part;     // [kWarps][rows_cap][kRB + 1]: the warps' sums of one pass
  float* h;        // [rows_cap][rk]: the block's sums
  uint16_t* term;  // [3][rows_cap][rk + 8]: the cluster's sums times the scale, as bf16 terms
  int pitch;       // rk + 8
};

size_t smem_bytes(int rows_cap, int rk) {
  return static_cast<size_t>(kWarps) * rows_cap * (kRB + 1) * 4 + static_cast<size_t>(rows_cap) * rk * 4 +
         static_cast<size_t>(3) * rows_cap * (rk + 8) * 2;
}

// Rows list[0 .. n) (n <= 16 MT) of adapter id.  Every block of the cluster calls it with the same arguments.
template <int MT>
__device__ void lora_rows(const LoraArgs& P, const Shared& S, const int* list, int n, int row0, int id,
                          cg::cluster_group& cluster) {
  const sf_lora_args& a = P.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int rank_c = static_cast<int>(cluster.block_rank());
  constexpr int ROWS = 16 * MT;

  // h: this warp's run of 64-channel steps
  const int steps = (a.K + 63) / 64, ways = kCluster * kWarps, w = rank_c * kWarps + warp;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * w / ways);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (w + 1) / ways);
  const uint16_t* xr[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int r = 16 * m + 8 * z + g;
      xr[m][z] = r < n ? a.x + static_cast<int64_t>(row0 + list[r]) * a.x_stride + 8 * t : nullptr;
    }
  const uint16_t* Aw = a.A + static_cast<int64_t>(id) * a.rank * a.K + 8 * t;
  for (int r0 = 0; r0 < a.rank; r0 += kRB) {
    float acc[MT][kRB / 8][4] = {};
    for (int s = s0; s < s1; ++s) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int k = 64 * s + 32 * half;
        const bool in = k + 8 * t < a.K;
        uint4 xv[MT][2], av[kRB / 8];
#pragma unroll
        for (int j = 0; j < kRB / 8; ++j) {
          const int r = r0 + 8 * j + g;
          av[j] = in && r < a.rank ? *reinterpret_cast<const uint4*>(Aw + static_cast<int64_t>(r) * a.K + k)
                                   : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int z = 0; z < 2; ++z)
            xv[m][z] = in && xr[m][z] ? *reinterpret_cast<const uint4*>(xr[m][z] + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < kRB / 8; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            bmma(acc[m][j], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, av[j].x, av[j].y);
            bmma(acc[m][j], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, av[j].z, av[j].w);
          }
      }
    }
    float* mine = S.part + warp * ROWS * (kRB + 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < kRB / 8; ++j)
#pragma unroll
        for (int z = 0; z < 4; ++z)
          mine[(16 * m + g + 8 * (z >> 1)) * (kRB + 1) + 8 * j + 2 * t + (z & 1)] = acc[m][j][z];
    __syncthreads();
    const int cols = min(kRB, P.rk - r0);
    for (int e = tid; e < ROWS * cols; e += kThreads) {
      const int r = e / cols, c = e - r * cols;
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += S.part[(v * ROWS + r) * (kRB + 1) + c];
      S.h[r * P.rk + r0 + c] = sum;
    }
    __syncthreads();
  }
  cluster.sync();
  const float scale = a.scale[id];
  for (int e = tid; e < ROWS * P.rk; e += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) sum += cluster.map_shared_rank(S.h, c)[e];
    float v = sum * scale;
    const int at = e / P.rk * S.pitch + e % P.rk;
#pragma unroll
    for (int z = 0; z < 3; ++z) {
      const __nv_bfloat16 b = __float2bfloat16_rn(v);
      S.term[z * ROWS * S.pitch + at] = __bfloat16_as_ushort(b);
      v -= __bfloat162float(b);
    }
  }
  __syncthreads();

  // out: this block's run of 8-column tiles
  const int tiles = (a.N + 7) / 8;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * rank_c / kCluster);
  const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (rank_c + 1) / kCluster);
  const uint16_t* Bw = a.B + static_cast<int64_t>(id) * a.N * a.rank + 4 * t;
  for (int tile = t0 + warp * kNB; tile < t1; tile += kWarps * kNB) {
    float acc[MT][kNB][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int r = 16 * m + 8 * z + g;
        const float* y = r < n && a.y ? a.y + static_cast<int64_t>(row0 + list[r]) * a.y_stride : nullptr;
#pragma unroll
        for (int j = 0; j < kNB; ++j) {
          const int c = 8 * (tile + j) + 2 * t;
          float2 v = make_float2(0.f, 0.f);
          if (y && tile + j < t1) {
            if (P.vec) {
              if (c < a.N) v = *reinterpret_cast<const float2*>(y + c);
            } else {
              if (c < a.N) v.x = y[c];
              if (c + 1 < a.N) v.y = y[c + 1];
            }
          }
          acc[m][j][2 * z] = v.x;
          acc[m][j][2 * z + 1] = v.y;
        }
      }
    float d[MT][kNB][4] = {};
    for (int k = 0; k < P.rk; k += 16) {
      uint2 b[kNB];
#pragma unroll
      for (int j = 0; j < kNB; ++j) {
        const int c = 8 * (tile + j) + g;
        b[j] = tile + j < t1 && c < a.N && k + 4 * t < a.rank
                   ? *reinterpret_cast<const uint2*>(Bw + static_cast<int64_t>(c) * a.rank + k)
                   : make_uint2(0, 0);
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int z = 2; z >= 0; --z) {  // the small terms first
          const uint16_t* from = S.term + (z * ROWS + 16 * m + g) * S.pitch + k + 4 * t;
          const uint2 lo = *reinterpret_cast<const uint2*>(from), hi = *reinterpret_cast<const uint2*>(from + 8 * S.pitch);
#pragma unroll
          for (int j = 0; j < kNB; ++j) bmma(d[m][j], lo.x, hi.x, lo.y, hi.y, b[j].x, b[j].y);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const int r = 16 * m + 8 * z + g;
        if (r >= n) continue;
        float* out = a.out + static_cast<int64_t>(row0 + list[r]) * a.out_stride;
#pragma unroll
        for (int j = 0; j < kNB; ++j) {
          const int c = 8 * (tile + j) + 2 * t;
          if (tile + j >= t1) continue;
          const float2 v = make_float2(acc[m][j][2 * z] + d[m][j][2 * z], acc[m][j][2 * z + 1] + d[m][j][2 * z + 1]);
          if (P.vec) {
            if (c < a.N) *reinterpret_cast<float2*>(out + c) = v;
          } else {
            if (c < a.N) out[c] = v.x;
            if (c + 1 < a.N) out[c + 1] = v.y;
          }
        }
      }
  }
  cluster.sync();  // the other blocks have read this one's sums
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 2)
lora_kernel(const __grid_constant__ LoraArgs P) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int ids[kWindow], list[kWindow], list_n;
  __shared__ unsigned leads[2];  // rows that are the first of their adapter
  const sf_lora_args& a = P.a;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x;
  Shared S;
  S.pitch = P.rk + 8;
  S.h = reinterpret_cast<float*>(smem);
  S.term = reinterpret_cast<uint16_t*>(S.h + P.rows_cap * P.rk);
  S.part = reinterpret_cast<float*>(S.term + 3 * P.rows_cap * S.pitch);
  const int task = blockIdx.x / kCluster, window = task / P.share, turn = task % P.share;
  const int row0 = window * kWindow, rows = min(kWindow, a.T - row0);
  if (tid < kWindow) {
    int id = -1;
    if (tid < rows) {
      int at = row0 + tid;
      if (a.row_of) at = a.row_of[at];
      if (at >= 0 && at < a.n_ids) id = a.ids[at];
      if (id < 0 || id >= a.n_adapters) id = -1;
    }
    ids[tid] = id;
  }
  __syncthreads();

  // Rows without an adapter.
  if (turn == 0 && a.out != a.y) {
    const int c0 = static_cast<int>(static_cast<int64_t>(a.N) * cluster.block_rank() / kCluster);
    const int c1 = static_cast<int>(static_cast<int64_t>(a.N) * (cluster.block_rank() + 1) / kCluster);
    for (int r = 0; r < rows; ++r) {
      if (ids[r] >= 0) continue;
      const float* y = a.y ? a.y + static_cast<int64_t>(row0 + r) * a.y_stride : nullptr;
      for (int c = c0 + tid; c < c1; c += kThreads)
        a.out[static_cast<int64_t>(row0 + r) * a.out_stride + c] = y ? y[c] : 0.f;
    }
  }

  // The window's adapters in the order of their first rows; this cluster takes every share-th.
  if (tid < kWindow) {
    bool first = ids[tid] >= 0;
    for (int q = 0; q < tid; ++q) first &= ids[q] != ids[tid];
    const unsigned m = __ballot_sync(0xffffffffu, first);
    if ((tid & 31) == 0) leads[tid >> 5] = m;
  }
  __syncthreads();
  unsigned long long lead = leads[0] | static_cast<unsigned long long>(leads[1]) << 32;
  for (int seen = 0; lead != 0; lead &= lead - 1, ++seen) {
    if (seen % P.share != turn) continue;
    const int id = ids[__ffsll(lead) - 1];
    if (tid < 32) {  // its rows
      int n = 0;
      for (int q = 0; q < kWindow; q += 32) {
        const unsigned m = __ballot_sync(0xffffffffu, ids[q + tid] == id);
        if (m >> tid & 1) list[n + __popc(m & ((1u << tid) - 1))] = q + tid;
        n += __popc(m);
      }
      if (tid == 0) list_n = n;
    }
    __syncthreads();
    const int n = list_n;
    for (int k = 0; k < n; k += 32) {
      if (n - k <= 16)
        lora_rows<1>(P, S, list + k, n - k, row0, id, cluster);
      else
        lora_rows<2>(P, S, list + k, min(32, n - k), row0, id, cluster);
    }
  }
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
  P.rk = (a->rank + 15) / 16 * 16;
  P.rows_cap = a->T <= 16 ? 16 : 32;
  P.vec = a->N % 2 == 0 && sf::aligned(a->out, 8) && a->out_stride % 2 == 0 &&
          (!a->y || (sf::aligned(a->y, 8) && a->y_stride % 2 == 0));
  // Two blocks an SM at least: with few windows, clusters share a window's adapters.
  const int windows = (a->T + kWindow - 1) / kWindow;
  P.share = std::max(1, std::min({kWindow, a->T, a->n_adapters, 2 * sf::sm_count() / kCluster / windows}));
  const size_t smem = smem_bytes(P.rows_cap, P.rk);
  if (smem > 48 * 1024)
    SF_CHECK_CUDA(
        cudaFuncSetAttribute(lora_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
  lora_kernel<<<windows * P.share * kCluster, kThreads, smem, sf::as_cuda(stream)>>>(P);
  return sf::check_launch("lora_kernel");
}
