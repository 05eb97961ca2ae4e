// sf_attn_paged: attention of a step's rows over a paged 4-bit KV cache.
#include <algorithm>
#include <cmath>

#include "paged.cuh"

namespace {

struct AttnArgs {
  const uint32_t *k_codes, *k_param, *v_codes, *v_param;
  const uint16_t* q;
  const int32_t *cu_rows, *len, *table;
  void* out;
  int64_t q_stride, out_stride, table_stride, page_rows;
  float scale;
  int T, R, Hq, Hkv, shift, num_pages, max_pages, window, bf16_out;
};

// A block per (row, query head); a warp per token, lane l holding dims
// [DL l, DL l + DL); online softmax per warp, the warps joined at the end.
constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attn_paged_row_kernel(const __grid_constant__ AttnArgs A) {
  constexpr int DL = D / 32;
  __shared__ int req_sh;
  __shared__ float m_sh[kWarps], l_sh[kWarps], o_sh[kWarps][D];
  const int t = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) req_sh = -1;
  __syncthreads();
  for (int i = tid; i < A.R; i += 32 * kWarps)
    if (A.cu_rows[i] <= t && t < A.cu_rows[i + 1]) req_sh = i;
  __syncthreads();
  const int i = req_sh;
  if (i < 0) return;
  const int h = hq / (A.Hq / A.Hkv);
  const int len = min(max(A.len[i], 0), A.max_pages << A.shift);
  const int pos = len - (A.cu_rows[i + 1] - t);
  const int end = pos + 1;
  const int begin = A.window > 0 ? max(0, pos - A.window + 1) : 0;
  float q[DL], o[DL];
#pragma unroll
  for (int j = 0; j < DL; ++j) {
    q[j] = sfd::bf16_bits_to_float(A.q[t * A.q_stride + hq * D + DL * lane + j]);
    o[j] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int tok = begin + warp; tok < end; tok += kWarps) {
    const int page = A.table[i * A.table_stride + (tok >> A.shift)];
    if (page < 0 || page >= A.num_pages) continue;
    const int64_t r = page * A.page_rows + (static_cast<int64_t>(h) << A.shift) + (tok & ((1 << A.shift) - 1));
    const uint32_t kp = A.k_param[r], vp = A.v_param[r];
    if ((kp & 0xffffu) == 0) continue;
    const float ks = sfd::half_bits_to_float(kp & 0xffff), kz = sfd::half_bits_to_float(kp >> 16);
    const float vs = sfd::half_bits_to_float(vp & 0xffff), vz = sfd::half_bits_to_float(vp >> 16);
    const uint32_t kw = A.k_codes[r * (D / 8) + DL * lane / 8] >> (4 * (DL * lane % 8));
    const uint32_t vw = A.v_codes[r * (D / 8) + DL * lane / 8] >> (4 * (DL * lane % 8));
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < DL; ++j) s = fmaf(q[j], static_cast<float>((kw >> (4 * j)) & 15u) - kz, s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= ks * A.scale;
    const float m2 = fmaxf(m, s), f = expf(m - m2), p = expf(s - m2);
    l = l * f + p;
#pragma unroll
    for (int j = 0; j < DL; ++j) o[j] = o[j] * f + p * vs * (static_cast<float>((vw >> (4 * j)) & 15u) - vz);
    m = m2;
  }
  if (lane == 0) {
    m_sh[warp] = m;
    l_sh[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < DL; ++j) o_sh[warp][DL * lane + j] = o[j];
  __syncthreads();
  float mm = -INFINITY;
  for (int w = 0; w < kWarps; ++w) mm = l_sh[w] == 0.f ? mm : fmaxf(mm, m_sh[w]);
  for (int x = tid; x < D; x += 32 * kWarps) {
    float sum = 0.f, ll = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      if (l_sh[w] == 0.f) continue;
      const float f = expf(m_sh[w] - mm);
      ll += l_sh[w] * f;
      sum += o_sh[w][x] * f;
    }
    const float v = ll == 0.f ? 0.f : sum / ll;
    const int64_t at = t * A.out_stride + hq * D + x;
    if (A.bf16_out)
      static_cast<__nv_bfloat16*>(A.out)[at] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(A.out)[at] = v;
  }
}

}  // namespace

extern "C" sf_status sf_attn_paged_workspace_size(int T, int R, int Hq, int Hkv, int d, size_t* bytes) {
  const char* what = "sf_attn_paged_workspace_size";
  SF_REQUIRE(bytes, "%s: null pointer", what);
  SF_REQUIRE(d == 64 || d == 128 || d == 256, "%s: d must be 64, 128 or 256", what);
  SF_REQUIRE(Hkv >= 1 && Hkv <= 256 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 64,
             "%s: need Hkv in [1, 256] and Hq/Hkv a whole number up to 64", what);
  SF_REQUIRE(T >= 0 && R >= 1 && R <= 8192, "%s: need T >= 0 and R in [1, 8192]", what);
  *bytes = 16;
  return SF_OK;
}

extern "C" sf_status sf_attn_paged(const sf_attn_paged_args* a, sf_stream_t stream) {
  const char* what = "sf_attn_paged";
  SF_REQUIRE(a, "%s: null arguments", what);
  sf_status st = sf::check_paged_kv(a->kv, what);
  if (st != SF_OK) return st;
  const sf_paged_kv& kv = *a->kv;
  size_t need = 0;
  st = sf_attn_paged_workspace_size(a->T, a->R, a->Hq, kv.Hkv, kv.d, &need);
  if (st != SF_OK) return st;
  SF_REQUIRE(a->max_pages >= 1 && static_cast<int64_t>(a->max_pages) * kv.page_size < (1ll << 31),
             "%s: need max_pages >= 1 and max_pages * page_size < 2^31", what);
  SF_REQUIRE(a->table_stride >= a->max_pages, "%s: table_stride is below max_pages", what);
  SF_REQUIRE(a->window >= 0, "%s: window must be >= 0", what);
  SF_REQUIRE(std::isfinite(a->scale), "%s: scale must be finite", what);
  SF_REQUIRE(a->out_type == SF_F32 || a->out_type == SF_BF16, "%s: out_type must be SF_F32 or SF_BF16", what);
  if (a->T == 0) return SF_OK;
  SF_REQUIRE(a->q && a->cu_rows && a->len && a->block_table && a->out && a->workspace, "%s: null pointer", what);
  const int64_t row = static_cast<int64_t>(a->Hq) * kv.d;
  SF_REQUIRE(a->q_stride >= row && a->out_stride >= row, "%s: q_stride and out_stride must be at least Hq * d", what);
  SF_REQUIRE(sf::aligned(a->q, 16) && a->q_stride % 8 == 0 && sf::aligned(a->out, 16) &&
                 a->out_stride % (a->out_type == SF_F32 ? 4 : 8) == 0,
             "%s: rows of q and out must be 16-byte aligned", what);
  SF_REQUIRE(sf::aligned(a->workspace, 16), "%s: workspace must be 16-byte aligned", what);
  SF_REQUIRE(a->ws_bytes >= need, "%s: workspace of %zu bytes is too small (need %zu)", what, a->ws_bytes, need);
  AttnArgs A{};
  A.k_codes = kv.k_codes;
  A.k_param = kv.k_param;
  A.v_codes = kv.v_codes;
  A.v_param = kv.v_param;
  A.q = a->q;
  A.cu_rows = a->cu_rows;
  A.len = a->len;
  A.table = a->block_table;
  A.out = a->out;
  A.q_stride = a->q_stride;
  A.out_stride = a->out_stride;
  A.table_stride = a->table_stride;
  A.page_rows = sf::page_rows(&kv);
  A.scale = a->scale;
  A.T = a->T;
  A.R = a->R;
  A.Hq = a->Hq;
  A.Hkv = kv.Hkv;
  A.shift = sf::log2i(kv.page_size);
  A.num_pages = kv.num_pages;
  A.max_pages = a->max_pages;
  A.window = a->window;
  A.bf16_out = a->out_type == SF_BF16;
  const dim3 grid(a->T, a->Hq);
  cudaStream_t s = sf::as_cuda(stream);
  if (kv.d == 64)
    attn_paged_row_kernel<64><<<grid, 32 * kWarps, 0, s>>>(A);
  else if (kv.d == 128)
    attn_paged_row_kernel<128><<<grid, 32 * kWarps, 0, s>>>(A);
  else
    attn_paged_row_kernel<256><<<grid, 32 * kWarps, 0, s>>>(A);
  return sf::check_launch("attn_paged_row_kernel");
}
