// The step's bookkeeping for a paged 4-bit KV cache (sf_paged_plan) and the
// append of its rows (sf_paged_append).
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include <cooperative_groups.h>

#include "launch.cuh"
#include "paged.cuh"
#include "produce.cuh"

namespace {

namespace cg = cooperative_groups;

// ---- sf_paged_plan ------------------------------------------------------------
//
// Three exclusive sums over the requests (rows added, pages taken, pages
// given back) decide everything: row r, the a-th page taken and the f-th page
// given back each find their request by a binary search in one of them.  The
// work is a few integers per row, so the kernel is bound by latency: one
// thread-block cluster does it all in one launch.  Every CTA of the cluster
// takes the sums over all requests itself (R <= 8192: three loads per request
// from L2, cheaper than an exchange), keeps them in shared memory, and does
// its share of the rows and pages.  The one cluster barrier separates every
// read of the lengths and the pushes onto the free list from the writes that
// may alias or follow them, so the lengths and the free count can be updated
// in place; what the rows need of a request after it is kept in shared memory.

constexpr int kPlanMaxR = 8192;

struct PlanArgs {
  sf_paged_plan_args a;
  int shift;  // log2(page_size)
  int vec;    // the rows' outputs allow 16-byte stores
  int own;    // rows a thread takes at a time: 1 or 4
};

// Index of the last entry of ascending cum[0..R] that is <= v (cum[0] = 0,
// v < cum[R]): the request that owns element v.
__device__ __forceinline__ int owner_of(const int* cum, int R, int v) {
  int lo = 0, hi = R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cum[mid] <= v)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Shared-memory integers per request: three sums, the tokens kept, the pages held.
constexpr int kPlanArrays = 5;

__global__ void __launch_bounds__(512) paged_plan_kernel(const __grid_constant__ PlanArgs P) {
  sfd::wait_for_previous();
  extern __shared__ int sh[];
  const sf_paged_plan_args& a = P.a;
  const int R = a.R, shift = P.shift, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  int* cu = sh;           // [R + 1] rows before request i
  int* ct = cu + R + 1;   // [R + 1] pages taken before it
  int* cb = ct + R + 1;   // [R + 1] pages given back before it
  int* kp = cb + R + 1;   // [R] tokens kept
  int* hv = kp + R;       // [R] pages held
  __shared__ long long part[32][3];
  __shared__ int bad_sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nthreads = nt * static_cast<int>(cluster.num_blocks());
  const int gtid = static_cast<int>(cluster.block_rank()) * nt + tid;
  if (tid == 0) bad_sh = 0;
  __syncthreads();

  // A thread's run of consecutive requests, their sums in 64 bits; lengths out
  // of range add nothing and are reported.
  const long long most = static_cast<long long>(a.max_pages) << shift;
  const int per = (R + nt - 1) / nt, r0 = min(tid * per, R), r1 = min(r0 + per, R);
  auto pages = [&](long long tokens) { return static_cast<int>((tokens + a.page_size - 1) >> shift); };
  long long s0 = 0, s1 = 0, s2 = 0;
  bool bad = false;
  for (int i = r0; i < r1; ++i) {
    const int len = a.len[i], keep = a.keep ? a.keep[i] : len, add = a.add[i];
    const long long now = static_cast<long long>(keep) + add;
    if (len < 0 || len > most || keep < 0 || keep > len || add < 0 || now > most) {
      bad = true;
      cu[i] = ct[i] = cb[i] = kp[i] = hv[i] = 0;
      continue;
    }
    const int have = pages(len), want = pages(now);
    cu[i] = add;
    ct[i] = max(want - have, 0);
    cb[i] = max(have - want, 0);
    kp[i] = keep;
    hv[i] = have;
    s0 += cu[i];
    s1 += ct[i];
    s2 += cb[i];
  }
  const int n_free = a.n_free[0];
  if (bad) bad_sh = 1;
  long long x0 = s0, x1 = s1, x2 = s2;  // inclusive over the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y0 = __shfl_up_sync(0xffffffffu, x0, o), y1 = __shfl_up_sync(0xffffffffu, x1, o),
                    y2 = __shfl_up_sync(0xffffffffu, x2, o);
    if (lane >= o) {
      x0 += y0;
      x1 += y1;
      x2 += y2;
    }
  }
  if (lane == 31) {
    part[warp][0] = x0;
    part[warp][1] = x1;
    part[warp][2] = x2;
  }
  __syncthreads();
  long long t0 = 0, t1 = 0, t2 = 0;
  for (int w = 0; w < (nt >> 5); ++w) {
    if (w == warp) {
      x0 += t0;
      x1 += t1;
      x2 += t2;
    }
    t0 += part[w][0];
    t1 += part[w][1];
    t2 += part[w][2];
  }
  int status = SF_PLAN_OK;
  if (n_free < 0 || n_free + t2 > a.free_cap || t1 > n_free + t2) status = SF_PLAN_PAGES;
  if (t0 > a.max_rows) status = SF_PLAN_ROWS;
  if (bad_sh) status = SF_PLAN_LENGTH;
  const bool ok = status == SF_PLAN_OK;
  if (ok) {  // then the sums fit 32 bits (max_rows, free_cap)
    int e0 = static_cast<int>(x0 - s0), e1 = static_cast<int>(x1 - s1), e2 = static_cast<int>(x2 - s2);
    for (int i = r0; i < r1; ++i) {
      const int add = cu[i], take = ct[i], back = cb[i];
      cu[i] = e0;
      ct[i] = e1;
      cb[i] = e2;
      e0 += add;
      e1 += take;
      e2 += back;
    }
    if (tid == 0) {
      cu[R] = static_cast<int>(t0);
      ct[R] = static_cast<int>(t1);
      cb[R] = static_cast<int>(t2);
    }
  }
  __syncthreads();
  const int rows = ok ? cu[R] : 0, taken = ok ? ct[R] : 0, given = ok ? cb[R] : 0;

  // Pages given back, on top of the free list: request i's last cb[i+1] - cb[i].
  for (int f = gtid; f < given; f += nthreads) {
    const int i = owner_of(cb, R, f);
    a.free_list[n_free + f] = a.block_table[i * a.table_stride + hv[i] - (cb[i + 1] - f)];
  }
  cluster.sync();

  const int top = n_free + given - 1;
  for (int i = gtid; i < R; i += nthreads) {
    a.len_out[i] = ok ? kp[i] + (cu[i + 1] - cu[i]) : a.len[i];
    a.cu_rows[i] = ok ? cu[i] : 0;
  }
  if (gtid == 0) {
    a.cu_rows[R] = rows;
    a.n_free_out[0] = n_free + given - taken;
    a.status[0] = status;
  }
  for (int k = gtid; k < taken; k += nthreads) {
    const int i = owner_of(ct, R, k);
    a.block_table[i * a.table_stride + hv[i] + (k - ct[i])] = a.free_list[top - k];
  }
  // Rows: with many, four consecutive ones a thread (one search, then a walk).
  const int own = P.own;
  for (int r0 = own * gtid; r0 < a.max_rows; r0 += own * nthreads) {
    int slot[4], pos[4], req[4];
    int i = r0 < rows ? owner_of(cu, R, r0) : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      slot[k] = req[k] = -1;
      pos[k] = 0;
      if (k >= own || r0 + k >= rows) continue;
      while (cu[i + 1] <= r0 + k) ++i;
      req[k] = i;
      pos[k] = kp[i] + (r0 + k - cu[i]);
      const int j = pos[k] >> shift;
      const int page = j < hv[i] ? a.block_table[i * a.table_stride + j] : a.free_list[top - (ct[i] + j - hv[i])];
      // (a page whose slots would not fit 32 bits is in no pool, and must not come out as another page's)
      if (page >= 0 && page <= INT_MAX >> shift) slot[k] = (page << shift) + (pos[k] & (a.page_size - 1));
    }
    if (P.vec && own == 4 && r0 + 4 <= a.max_rows) {
      *reinterpret_cast<int4*>(a.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.row_request + r0) = make_int4(req[0], req[1], req[2], req[3]);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < own && r0 + k < a.max_rows) {
          a.slots[r0 + k] = slot[k];
          a.positions[r0 + k] = pos[k];
          a.row_request[r0 + k] = req[k];
        }
    }
  }
}

// ---- sf_paged_append ----------------------------------------------------------
//
// A half warp per (row, head), so that what is done once per token-head is
// shared by two: its lane l holds the pairs (i, i + d/2) for i in [NP l, NP l +
// NP), NP = d/32, so a rotation needs no exchange, the group's min and max are a
// butterfly over 16 lanes, and the lanes of a code word OR their codes
// together.  theta^(-2i/d) is taken once per block, the sines and cosines of a
// group of rows once per block by all its threads, shared by the rows' heads.
//
// Every result is the fp64 or IEEE one rounded once, as sf_rope and
// sf_kv_append have it, but computed in fp32 where that cannot differ, with one
// rare branch per token-head for where it might:
//  * a query is rotated in fp32 and both ends of its error interval rounded to
//    bf16; where they differ (one entry in some thousands) fp64 decides.  The
//    conversions to and from fp64 of every query bound the kernel before;
//  * a scale is (max - min) / 15 rounded to fp32, then fp16: times 1/15, unless
//    that lies within 4 units of an fp16 midpoint;
//  * a code is rint(x / s): x times a reciprocal, unless that lies within 2^-16
//    of a half.
// Bound by memory for many rows (a source value is read once, 4 bits and a bf16
// come out), so a warp has the sources of the next kAhead rows of its heads on
// their way; by latency for few rows, when a row's heads are spread over
// blocks.

constexpr int kAppWarps = 8;

struct AppendArgs {
  const void *k, *v, *q;
  uint16_t *q_out, *k_val, *v_val;
  uint32_t *k_codes, *k_param, *v_codes, *v_param;
  const int32_t *slots, *positions;
  int64_t k_stride, v_stride, q_stride, q_out_stride, page_rows;
  double theta;
  int T, Hq, Hkv, shift, slot_end;
  int group;  // rows that a block takes at a time
};

template <int NP, typename S>
__device__ __forceinline__ void load_row(const S* p, float (&x)[NP]) {
  if constexpr (sizeof(S) == 4) {
    if constexpr (NP == 2) {
      *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(p);
    } else {
#pragma unroll
      for (int j = 0; j < NP; j += 4) *reinterpret_cast<float4*>(x + j) = *reinterpret_cast<const float4*>(p + j);
    }
  } else {
    uint32_t u[NP / 2];
    if constexpr (NP == 2)
      u[0] = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (NP == 4)
      *reinterpret_cast<uint2*>(u) = *reinterpret_cast<const uint2*>(p);
    else
      *reinterpret_cast<uint4*>(u) = *reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int j = 0; j < NP; j += 2) {
      x[j] = __uint_as_float(u[j / 2] << 16);
      x[j + 1] = __uint_as_float(u[j / 2] & 0xFFFF0000u);
    }
  }
}

// NP bf16 as NP / 2 words.
template <int NP>
__device__ __forceinline__ void store_bf16(uint16_t* p, const uint32_t (&u)[NP / 2]) {
  if constexpr (NP == 2)
    *reinterpret_cast<uint32_t*>(p) = u[0];
  else if constexpr (NP == 4)
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return reinterpret_cast<const uint32_t&>(v);
}

// (max - min) / 15 as sf_kv_append rounds it; at least the smallest fp16, 1 for 0.
__device__ __forceinline__ float scale_of(float span) {
  float q = span * (1.f / 15.f);  // within 2 units of the quotient
  const uint32_t low = __float_as_uint(q) & 0x1FFFu;
  if (q < 6.2e-5f || low - 0xFFCu <= 8u) q = __fdiv_rn(span, 15.0f);  // fp16's subnormals, or near a midpoint
  const float s = __half2float(__float2half_rn(fminf(q, 65504.0f)));
  return s == 0.f ? 1.f : s;
}

// rint(x / s) from x times 1/s; near: too close to a half (or so large that the sum below no longer rounds, or to
// count: beyond 2^7 the product's error is).
__device__ __forceinline__ float quotient(float x, float inv, bool& near) {
  const float r = x * inv, n = (r + 12582912.f) - 12582912.f;
  near |= !(fabsf(r - n) <= 0.5f - 0x1p-16f) || fabsf(r) > 64.f;
  return n;
}

template <int D, typename S>
__global__ void __launch_bounds__(32 * kAppWarps) paged_append_kernel(const __grid_constant__ AppendArgs A) {
  constexpr int NP = D / 32, H = D / 2, MAX_ROWS = 32 * kAppWarps / H, kAhead = 8 / NP < 2 ? 1 : 2;
  __shared__ double freq[H];
  __shared__ double2 turn[2][MAX_ROWS][H];  // cosine, sine; two groups, so that one barrier a group does
  __shared__ float2 turn32[2][MAX_ROWS][H];
  sfd::wait_for_previous();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool rot = A.theta > 0.0;
  if (rot && tid < H) freq[tid] = pow(A.theta, -2.0 * tid / D);
  __syncthreads();
  // pairs of heads: of keys, of values, of queries
  const int kv_pairs = (A.Hkv + 1) / 2, units = 2 * kv_pairs + (A.Hq + 1) / 2, step = gridDim.y * kAppWarps;
  const int half = lane >> 4, hl = lane & 15;
  int buf = 0;
  for (int row0 = blockIdx.x * A.group; row0 < A.T; row0 += gridDim.x * A.group, buf ^= 1) {
    const int rows = min(A.group, A.T - row0);
    float next_lo[kAhead][NP], next_hi[kAhead][NP];
    int next_slot[kAhead];
    auto load = [&](int u, int k0) {  // rows k0 .. of the group
      const int kind = u < kv_pairs ? 0 : u < 2 * kv_pairs ? 1 : 2, h = 2 * (u - kind * kv_pairs) + half;
      const bool in = h < (kind == 2 ? A.Hq : A.Hkv);
      const int64_t stride = kind == 0 ? A.k_stride : kind == 1 ? A.v_stride : A.q_stride;
      const S* src = static_cast<const S*>(kind == 0 ? A.k : kind == 1 ? A.v : A.q) + (row0 + k0) * stride + h * D +
                     NP * hl;
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        next_slot[k] = -1;
        if (k0 + k >= rows) continue;
        next_slot[k] = A.slots[row0 + k0 + k];
        if (!in) continue;
        load_row<NP, S>(src + k * stride, next_lo[k]);
        load_row<NP, S>(src + k * stride + H, next_hi[k]);
      }
    };
    // a warp takes every step-th (unit, kAhead rows) of the group, the units of the first rows first
    int u = blockIdx.y * kAppWarps + warp, k0 = 0;
    auto wrap = [&]() {
      for (; u >= units && k0 < rows; u -= units) k0 += kAhead;
    };
    wrap();
    if (k0 < rows) load(u, k0);
    if (rot) {
      if (tid < rows * H) {
        double s, c;
        sincos(A.positions[row0 + tid / H] * freq[tid % H], &s, &c);
        turn[buf][tid / H][tid % H] = make_double2(c, s);
        turn32[buf][tid / H][tid % H] = make_float2(static_cast<float>(c), static_cast<float>(s));
      }
      __syncthreads();
    }
    while (k0 < rows) {
      float lo[kAhead][NP], hi[kAhead][NP];
      int slots[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        slots[k] = next_slot[k];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          lo[k][j] = next_lo[k][j];
          hi[k][j] = next_hi[k][j];
        }
      }
      const int kind = u < kv_pairs ? 0 : u < 2 * kv_pairs ? 1 : 2;  // keys, values, queries
      const int h = 2 * (u - kind * kv_pairs) + half, row_k = k0;
      const bool in = h < (kind == 2 ? A.Hq : A.Hkv);  // an odd number of heads leaves half a warp over
      u += step;
      wrap();
      if (k0 < rows) load(u, k0);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int slot = slots[k], row = row_k + k;
        if (slot < 0 || slot >= A.slot_end) continue;  // the same for the whole warp
        const int64_t t = row0 + row;
        if (kind == 2) {
          if (!in) continue;
          // In fp32 with cosine and sine rounded to it: the two products are off by 2^-23 of themselves, the sum by
          // 2^-24 of itself, together within e.
          uint32_t o[2][NP / 2];
          bool near = false;
#pragma unroll
          for (int j = 0; j < NP; j += 2) {
            float v[2][2], e[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float2 cs = turn32[buf][row][NP * hl + j + i];
              const float x = lo[k][j + i], y = hi[k][j + i];
              v[0][i] = fmaf(x, cs.x, -(y * cs.y));
              v[1][i] = fmaf(x, cs.y, y * cs.x);
              e[i] = fmaf(fabsf(x) + fabsf(y), 0x1p-22f, 1e-40f);  // |cosine|, |sine| <= 1
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              o[z][j / 2] = pack_bf16(v[z][0] - e[0], v[z][1] - e[1]);
              near |= o[z][j / 2] != pack_bf16(v[z][0] + e[0], v[z][1] + e[1]);
            }
          }
          if (near) {
#pragma unroll
            for (int j = 0; j < NP; ++j) {
              const double2 cs = turn[buf][row][NP * hl + j];
              const double x = lo[k][j], y = hi[k][j];
              const uint32_t a = sfd::to_bf16(x * cs.x - y * cs.y), b = sfd::to_bf16(y * cs.x + x * cs.y);
              o[0][j / 2] = (j & 1) ? (o[0][j / 2] | a << 16) : a;
              o[1][j / 2] = (j & 1) ? (o[1][j / 2] | b << 16) : b;
            }
          }
          uint16_t* out = A.q_out + t * A.q_out_stride + h * D + NP * hl;
          store_bf16<NP>(out, o[0]);
          store_bf16<NP>(out + H, o[1]);
          continue;
        }
        if (rot && kind == 0) {
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            const double2 cs = turn[buf][row][NP * hl + j];
            const double x = lo[k][j], y = hi[k][j];
            lo[k][j] = static_cast<float>(x * cs.x - y * cs.y);
            hi[k][j] = static_cast<float>(y * cs.x + x * cs.y);
          }
        }
        // 4-bit min-max quantization of the token-head
        float mn = fminf(lo[k][0], hi[k][0]), mx = fmaxf(lo[k][0], hi[k][0]);
#pragma unroll
        for (int j = 1; j < NP; ++j) {
          mn = fminf(mn, fminf(lo[k][j], hi[k][j]));
          mx = fmaxf(mx, fmaxf(lo[k][j], hi[k][j]));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
        const float s = scale_of(__fsub_rn(mx, mn));
        float inv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
        bool near = false;
        float zf = quotient(-mn, inv, near), c[2][NP];
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          c[0][j] = quotient(lo[k][j], inv, near);
          c[1][j] = quotient(hi[k][j], inv, near);
        }
        if (near) {
          zf = rintf(__fdiv_rn(-mn, s));
#pragma unroll
          for (int j = 0; j < NP; ++j) {
            c[0][j] = rintf(__fdiv_rn(lo[k][j], s));
            c[1][j] = rintf(__fdiv_rn(hi[k][j], s));
          }
        }
        zf = fminf(fmaxf(zf, 0.f), 15.f);
        uint32_t wl = 0, wh = 0;  // the lane's codes, then at their place in the word
#pragma unroll
        for (int j = 0; j < NP; ++j) {
          c[0][j] = fminf(fmaxf(c[0][j] + zf, 0.f), 15.f);
          c[1][j] = fminf(fmaxf(c[1][j] + zf, 0.f), 15.f);
          wl |= (__float_as_uint(c[0][j] + 8388608.f) & 15u) << (4 * j);
          wh |= (__float_as_uint(c[1][j] + 8388608.f) & 15u) << (4 * j);
        }
        if constexpr (NP < 8) {
          wl <<= 4 * (NP * hl & 7);
          wh <<= 4 * (NP * hl & 7);
        }
#pragma unroll
        for (int o = 1; o < 8 / NP; o <<= 1) {
          wl |= __shfl_xor_sync(0xffffffffu, wl, o);
          wh |= __shfl_xor_sync(0xffffffffu, wh, o);
        }
        if (!in) continue;  // the whole warp has shuffled
        const int64_t r = (slot >> A.shift) * A.page_rows + (h << A.shift) + (slot & ((1 << A.shift) - 1));
        uint32_t* codes = (kind ? A.v_codes : A.k_codes) + r * (D / 8);
        if (NP == 8 || hl % (8 / NP) == 0) {
          codes[NP * hl / 8] = wl;
          codes[H / 8 + NP * hl / 8] = wh;
        }
        if (hl == 0)
          (kind ? A.v_param : A.k_param)[r] =
              static_cast<uint32_t>(__half_as_ushort(__float2half_rn(s))) |
              static_cast<uint32_t>(__half_as_ushort(__float2half_rn(zf))) << 16;
        uint16_t* val = kind ? A.v_val : A.k_val;
        if (val != nullptr) {
          uint32_t o[2][NP / 2];
#pragma unroll
          for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int j = 0; j < NP; j += 2) o[z][j / 2] = pack_bf16(s * (c[z][j] - zf), s * (c[z][j + 1] - zf));
          val += (t * A.Hkv + h) * D + NP * hl;
          store_bf16<NP>(val, o[0]);
          store_bf16<NP>(val + H, o[1]);
        }
      }
    }
  }
}

using AppendKernel = void (*)(AppendArgs);

template <typename S>
AppendKernel append_kernel(int d) {
  return d == 64 ? paged_append_kernel<64, S> : d == 128 ? paged_append_kernel<128, S> : paged_append_kernel<256, S>;
}

}  // namespace

extern "C" sf_status sf_paged_plan(const sf_paged_plan_args* a, sf_stream_t stream) {
  SF_REQUIRE(a, "sf_paged_plan: null arguments");
  SF_REQUIRE(a->len && a->add && a->block_table && a->free_list && a->n_free && a->len_out && a->n_free_out &&
                 a->cu_rows && a->slots && a->positions && a->row_request && a->status,
             "sf_paged_plan: null pointer");
  SF_REQUIRE(a->R >= 1 && a->R <= kPlanMaxR, "sf_paged_plan: R must be in [1, %d]", kPlanMaxR);
  SF_REQUIRE(sf::pow2_in(a->page_size, 16, 256), "sf_paged_plan: page_size must be a power of two in [16, 256]");
  SF_REQUIRE(a->max_pages >= 1 && static_cast<int64_t>(a->max_pages) * a->page_size < (1ll << 31),
             "sf_paged_plan: need max_pages >= 1 and max_pages * page_size < 2^31");
  SF_REQUIRE(a->table_stride >= a->max_pages, "sf_paged_plan: table_stride is below max_pages");
  // (the loops' indexes run past the two by less than that)
  SF_REQUIRE(a->max_rows >= 1 && a->free_cap >= 1 && a->max_rows <= 1 << 30 && a->free_cap <= 1 << 30,
             "sf_paged_plan: max_rows and free_cap must be in [1, 2^30]");
  PlanArgs P{*a, sf::log2i(a->page_size),
             sf::aligned(a->slots, 16) && sf::aligned(a->positions, 16) && sf::aligned(a->row_request, 16),
             a->max_rows > 4096 ? 4 : 1};
  // One small block for a decode batch; sixteen blocks share the rows of a step
  // that has many (1000 requests, 65536 rows: 10 us; 13 with eight of 1024 threads).
  const bool small = a->R <= 128 && a->max_rows <= 512;
  const int blocks = small || a->max_rows <= 4096 ? 1 : 16;
  auto smem_for = [](int R) { return static_cast<size_t>(kPlanArrays) * (R + 1) * sizeof(int); };
  static std::atomic<unsigned long long> told{0};
  const sf_status st = sf::allow_smem(paged_plan_kernel, smem_for(kPlanMaxR), told, true);
  if (st != SF_OK) return st;
  return sf::launch("paged_plan_kernel", paged_plan_kernel, dim3(blocks), small ? 128 : 512, smem_for(a->R), blocks,
                    sf::as_cuda(stream), P);
}

extern "C" sf_status sf_paged_append(const sf_paged_append_args* a, sf_stream_t stream) {
  const char* what = "sf_paged_append";
  SF_REQUIRE(a, "%s: null arguments", what);
  sf_status st = sf::check_paged_kv(a->kv, what);
  if (st != SF_OK) return st;
  const sf_paged_kv& kv = *a->kv;
  SF_REQUIRE(a->T >= 0, "%s: T must be >= 0", what);
  SF_REQUIRE(a->src_type == SF_F32 || a->src_type == SF_BF16, "%s: src_type must be SF_F32 or SF_BF16", what);
  SF_REQUIRE(a->Hq >= 0 && a->Hq <= 1024, "%s: Hq must be in [0, 1024]", what);
  SF_REQUIRE(a->theta >= 0.0 && std::isfinite(a->theta), "%s: theta must be finite and >= 0", what);
  SF_REQUIRE(a->theta > 0.0 || a->Hq == 0, "%s: q is only rotated: it needs theta > 0", what);
  if (a->T == 0) return SF_OK;  // (tensors without elements have no address)
  SF_REQUIRE((a->q != nullptr) == (a->Hq > 0) && (a->q_out != nullptr) == (a->Hq > 0),
             "%s: q and q_out go with Hq > 0", what);
  SF_REQUIRE(a->k && a->v && a->slots, "%s: null pointer", what);
  SF_REQUIRE(a->theta == 0.0 || a->positions, "%s: the rotation needs positions", what);
  const int es = a->src_type == SF_F32 ? 4 : 2;
  const int64_t kv_row = static_cast<int64_t>(kv.Hkv) * kv.d, q_row = static_cast<int64_t>(a->Hq) * kv.d;
  SF_REQUIRE(a->k_stride >= kv_row && a->v_stride >= kv_row, "%s: k_stride and v_stride must be at least Hkv * d",
             what);
  SF_REQUIRE(a->Hq == 0 || (a->q_stride >= q_row && a->q_out_stride >= q_row),
             "%s: q_stride and q_out_stride must be at least Hq * d", what);
  auto rows16 = [](const void* p, int64_t stride, int size) {
    return sf::aligned(p, 16) && stride * size % 16 == 0;
  };
  SF_REQUIRE(rows16(a->k, a->k_stride, es) && rows16(a->v, a->v_stride, es) &&
                 (a->Hq == 0 || (rows16(a->q, a->q_stride, es) && rows16(a->q_out, a->q_out_stride, 2))),
             "%s: rows of k, v, q and q_out must be 16-byte aligned", what);
  SF_REQUIRE((!a->k_val || sf::aligned(a->k_val, 16)) && (!a->v_val || sf::aligned(a->v_val, 16)),
             "%s: k_val and v_val must be 16-byte aligned", what);
  AppendArgs A{};
  A.k = a->k;
  A.v = a->v;
  A.q = a->q;
  A.q_out = a->q_out;
  A.k_val = a->k_val;
  A.v_val = a->v_val;
  A.k_codes = kv.k_codes;
  A.k_param = kv.k_param;
  A.v_codes = kv.v_codes;
  A.v_param = kv.v_param;
  A.slots = a->slots;
  A.positions = a->positions;
  A.k_stride = a->k_stride;
  A.v_stride = a->v_stride;
  A.q_stride = a->q_stride;
  A.q_out_stride = a->q_out_stride;
  A.page_rows = sf::page_rows(&kv);
  A.theta = a->theta;
  A.T = a->T;
  A.Hq = a->Hq;
  A.Hkv = kv.Hkv;
  A.shift = sf::log2i(kv.page_size);
  A.slot_end = kv.num_pages * kv.page_size;
  // One round of blocks that fit the SMs.  Few rows: a row's heads are spread over blocks.  Many rows: a block keeps
  // all heads of a group of rows (as many as its threads have sines for, as few as make one round, an even number
  // where a warp takes two at a time) and loops over groups, so that what a block does once is done less often (us; one
  // row a group and blocks for two or three rounds: 1000 rows of 40 rotated heads of 128, 11.2 / 13.3; 1000 of 12 of
  // 64, 4.7 / 5.9).
  const AppendKernel kernel = a->src_type == SF_F32 ? append_kernel<float>(kv.d) : append_kernel<uint16_t>(kv.d);
  static std::atomic<int> fits[2][3];  // the kernels' blocks on an SM, once asked for
  std::atomic<int>& known = fits[a->src_type == SF_F32][kv.d / 128];
  int fit = known.load(std::memory_order_relaxed);
  if (fit == 0) {
    SF_CHECK_CUDA(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kernel, 32 * kAppWarps, 0));
    known.store(fit, std::memory_order_relaxed);
  }
  const int sms = sf::sm_count(), room = sms * std::max(fit, 1), most = 64 * kAppWarps / kv.d;
  A.group = std::min(most, (a->T - 1) / room + 1);
  if (A.group > 1 && kv.d < 256) A.group += A.group % 2;
  const int need = ((kv.Hkv + 1) / 2 * 2 + (a->Hq + 1) / 2 + kAppWarps - 1) / kAppWarps;  // blocks that one row can fill
  const int gx = std::min((a->T - 1) / A.group + 1, room);
  const int gy = std::max(1, std::min(need, sms * 2 / gx));
  return sf::launch("paged_append_kernel", kernel, dim3(gx, gy), 32 * kAppWarps, 0, 1, sf::as_cuda(stream), A);
}
