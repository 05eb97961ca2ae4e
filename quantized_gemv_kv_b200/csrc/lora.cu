// sf_lora_add: low-rank adapters of many requests beside a shared projection,
//   out[t] = y[t] + scale_a B_a (A_a x[t]),  a the adapter of row t.
#include <algorithm>

#include "sf_internal.h"

namespace {

constexpr int kLoraMaxRank = 128;
constexpr int kWarps = 8;

// A block per row: a warp per rank row of A_a, then a thread per output.
__global__ void __launch_bounds__(32 * kWarps) lora_row_kernel(const __grid_constant__ sf_lora_args a) {
  __shared__ float h[kLoraMaxRank];
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int at = t, id = -1;
  if (a.row_of) at = a.row_of[t];
  if (at >= 0 && at < a.n_ids) id = a.ids[at];
  if (id < 0 || id >= a.n_adapters) id = -1;
  if (id >= 0) {
    const uint16_t* x = a.x + t * a.x_stride;
    for (int r = warp; r < a.rank; r += kWarps) {
      const uint16_t* A = a.A + (static_cast<int64_t>(id) * a.rank + r) * a.K;
      float s = 0.f;
      for (int k = lane; k < a.K; k += 32) s = fmaf(sfd::bf16_bits_to_float(A[k]), sfd::bf16_bits_to_float(x[k]), s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) h[r] = s;
    }
    __syncthreads();
  }
  const float sc = id >= 0 ? a.scale[id] : 0.f;
  for (int n = tid; n < a.N; n += 32 * kWarps) {
    float v = a.y ? a.y[t * a.y_stride + n] : 0.f;
    if (id >= 0) {
      const uint16_t* B = a.B + (static_cast<int64_t>(id) * a.N + n) * a.rank;
      float s = 0.f;
      for (int r = 0; r < a.rank; ++r) s = fmaf(sfd::bf16_bits_to_float(B[r]), h[r], s);
      v = fmaf(sc, s, v);
    }
    a.out[t * a.out_stride + n] = v;
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
  lora_row_kernel<<<a->T, 32 * kWarps, 0, sf::as_cuda(stream)>>>(*a);
  return sf::check_launch("lora_row_kernel");
}
