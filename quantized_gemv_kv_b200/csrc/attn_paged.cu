// sf_attn_paged: attention of a step's rows over a paged 4-bit KV cache.
#include <climits>
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

// How the work is laid out.  A request's rows times the query heads of one KV
// head are the columns that read the same keys; a column block takes COLS = 8
// NT of them.  A segment is one (request, column block, KV head); its tokens
// come in stages of TOK.  Stages of all segments, in order, are the units,
// and every block (and in it every warp) takes an equal run of them, so a
// 128K-token request and a hundred short ones fill the SMs alike.  A segment
// that lies within one warp's run is written by it; the parts of one that does
// not are joined in shared memory, and across blocks by a second kernel.
//
// A warp's stage of 16-token tiles:
//  * scores: mma.m16n8k32 (s8), rows = tokens, columns = query columns.  A
//    4-bit code word is two operand registers by a mask and a shift, so no
//    conversion is needed; q enters as X = rint(q 2^(21-e)) (e the exponent of
//    its row's largest entry) in three balanced base-256 digits, one product
//    each, exact in 32-bit integers.  The accumulators start from -8 sum X, so
//    they hold sum X (c - 8), and the rest of the zero point is (z - 8) sum X;
//  * online softmax in base 2, one maximum per column and stage;
//  * values: mma.m16n8k16 (f16), rows = dims, columns = query columns, k =
//    tokens.  A byte permute pairs the codes of two tokens, a mask-and-or makes
//    them 1024 + c and 1024 + 16 c, and one exact f16 operation c - 8, so the
//    sums carry no offset.  The weights p v_s enter as an f16 value and its f16
//    remainder (22 bits; v_s scaled by a power of two that follows the largest
//    seen), which the columns' transposed scores become by movmatrix.
// The k index of the value product is free, so the tokens of a tile are
// ordered such that both fragment loads are free of bank conflicts.
//
// The cache streams through a ring of STAGES stages per warp (cp.async, no
// barrier between warps), two stages ahead across segment ends, the block
// table's entries a stage ahead of that.

// log2(e)
constexpr float kLog2e = 1.4426950408889634f;

template <int D_, int NT_, int TOK_, int WARPS_, int STAGES_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, TOK = TOK_, WARPS = WARPS_, STAGES = STAGES_;
  static constexpr int COLS = 8 * NT, TILES = TOK / 16, GROUPS = TOK / 16;
  static constexpr int KW = D / 32, VW = D / 64, MT = D / 16;  // words per lane of a K row, of a V row; dim tiles
  static constexpr int ROWB = D / 2, TILEB = 16 * ROWB, CH = D / 32;  // bytes of a row and of a tile; 16-byte chunks
  static constexpr int PAR = 2 * TOK * ROWB;                          // offset of the params in a stage
  static constexpr int STAGEB = PAR + 2 * TOK * 4;
  static constexpr int PART = COLS * (D + 1);  // floats of one partial: the columns' outputs, then their log sums
  static constexpr int RINGB = STAGES * STAGEB;
  static constexpr int SMEM = WARPS * (RINGB + PART * 4);  // the rings, then a partial for each warp
  static_assert(PART * 4 <= RINGB, "a warp's second partial takes its ring's place");
  static_assert(SMEM <= 220 * 1024, "shared memory");
};

// Offset in a 16-token tile of chunk ch (16 bytes) of row r: rows k and k + 4
// (a K load's quarter warp) and rows 4j .. 4j + 3 (a V load's) meet no bank twice.
template <int D>
__device__ __forceinline__ int swz(int r, int ch) {
  if constexpr (D == 64) return ((r & ~3) | ((r & 3) ^ (2 * ((r >> 2) & 1)))) * 32 + ch * 16;
  if constexpr (D == 128)
    return (r >> 1) * 128 + (((r & 1) ^ ((r >> 2) & 1)) * 64) + ((ch ^ (2 * ((r >> 1) & 1))) * 16);
  return r * 128 + ((ch ^ ((2 * (r & 3)) | ((r >> 2) & 1))) * 16);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(bytes));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void imma(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1, int c0, int c1, int c2, int c3) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}

__device__ __forceinline__ void hmma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The low (shift 0) and high nibbles of bytes 0 and 2 of x as f16 c - 8.
__device__ __forceinline__ uint32_t nib_lo(uint32_t x) {
  const uint32_t v = (x & 0x000F000Fu) | 0x64006400u;  // 1024 + c
  const __half2 r = __hsub2(reinterpret_cast<const __half2&>(v), __float2half2_rn(1032.f));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t x) {
  const uint32_t v = (x & 0x00F000F0u) | 0x64006400u;  // 1024 + 16 c
  const __half2 r =
      __hfma2(reinterpret_cast<const __half2&>(v), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  return reinterpret_cast<const uint32_t&>(r);
}

// One request's columns and stages.
struct Req {
  int row0, rows;    // its rows in q and out (those below T)
  int last;          // cu_rows[i + 1]: row t is the token at len - (last - t)
  int len, end;      // tokens held; tokens that its last row sees
  int st0, stages;   // first stage, number of stages (at least 1)
  int segs;          // segments
};

template <class C>
__device__ __forceinline__ Req load_req(const AttnArgs& A, int i) {
  Req q;
  const int c0 = A.cu_rows[i];
  q.last = A.cu_rows[i + 1];
  q.row0 = max(c0, 0);
  q.rows = max(min(q.last, A.T) - q.row0, 0);
  q.len = min(max(A.len[i], 0), A.max_pages << A.shift);
  q.end = max(q.len - (q.last - (q.row0 + q.rows)), 0);
  const int first = q.len - (q.last - q.row0);  // the first row's position
  q.st0 = A.window > 0 ? max(first - A.window + 1, 0) / C::TOK : 0;
  q.stages = max((q.end + C::TOK - 1) / C::TOK - q.st0, 1);
  q.segs = (q.rows * (A.Hq / A.Hkv) + C::COLS - 1) / C::COLS * A.Hkv;
  return q;
}

// A place in the run of units.
struct Cursor {
  Req q;
  int i, seg, tile;
};

template <class C>
__device__ __forceinline__ void advance(const AttnArgs& A, Cursor& c) {
  if (++c.tile < c.q.stages) return;
  c.tile = 0;
  if (++c.seg < c.q.segs) return;
  c.seg = 0;
  do {
    ++c.i;
    if (c.i >= A.R) return;
    c.q = load_req<C>(A, c.i);
  } while (c.q.segs == 0);
}

// What the second kernel needs of a block: the segment that starts in it and
// ends in a later block.
struct Tail {
  int open;      // 1: there is one
  int i, seg;    // which
  int last_cta;  // the block that holds its last unit
};

struct Work {
  AttnArgs a;
  Tail* tails;    // [blocks]
  float* parts;   // [blocks][2][PART]: a block's part of a segment begun earlier (0), of its open one (1)
  int blocks;
};

// Where run c of n equal runs of u units begins, and the run that holds unit x.
__device__ __forceinline__ long long run_begin(long long u, int n, int c) { return u * c / n; }
__device__ __forceinline__ int run_of(long long u, int n, long long x) {
  return static_cast<int>(((x + 1) * n - 1) / u);
}

template <class C>
__device__ __forceinline__ void put(const AttnArgs& A, const Req& q, int seg, int col, int x, float v0, float v1) {
  // dims x, x + 1 of column col of segment seg
  const int g = A.Hq / A.Hkv, c = seg / A.Hkv * C::COLS + col;
  if (c >= q.rows * g) return;
  const int64_t at = (q.row0 + c / g) * A.out_stride + static_cast<int64_t>(seg % A.Hkv * g + c % g) * C::D + x;
  if (A.bf16_out)
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(A.out) + at) = __floats2bfloat162_rn(v0, v1);
  else
    *reinterpret_cast<float2*>(static_cast<float*>(A.out) + at) = make_float2(v0, v1);
}

template <class C>
__global__ void __launch_bounds__(32 * C::WARPS, 1) attn_paged_kernel(const __grid_constant__ Work W) {
  constexpr int D = C::D, NT = C::NT, TOK = C::TOK, TILES = C::TILES, KW = C::KW, VW = C::VW, MT = C::MT;
  constexpr int NTHR = 32 * C::WARPS;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long pre[NTHR + 1];  // units before each thread's run of requests
  __shared__ long long wsum[C::WARPS];
  struct Part {
    long long us, ue;  // the segment's units; us < 0: none
    int i, seg;
  };
  __shared__ Part parts[C::WARPS][2];
  const AttnArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int group = A.Hq / A.Hkv;

  // The units of all requests.
  const int per = (A.R + NTHR - 1) / NTHR;
  long long mine = 0;
  for (int i = min(tid * per, A.R); i < min((tid + 1) * per, A.R); ++i) {
    const Req q = load_req<C>(A, i);
    mine += static_cast<long long>(q.segs) * q.stages;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[warp] = x;
  if (lane < 2) parts[warp][lane].us = -1;
  __syncthreads();
  long long before = 0, units = 0;
#pragma unroll
  for (int w = 0; w < C::WARPS; ++w) {
    if (w < warp) before += wsum[w];
    units += wsum[w];
  }
  pre[tid] = before + x - mine;
  if (tid == 0) pre[NTHR] = units;
  __syncthreads();

  // This block's run of units, then this warp's.  A block that has work has
  // at least a unit for each warp, if there are that many.
  const int blocks = static_cast<int>(min(static_cast<long long>(W.blocks), (units + C::WARPS - 1) / C::WARPS));
  if (static_cast<int>(blockIdx.x) >= blocks) {
    if (tid == 0 && static_cast<int>(blockIdx.x) < W.blocks) W.tails[blockIdx.x].open = 0;
    return;
  }
  const long long b_lo = run_begin(units, blocks, blockIdx.x), b_hi = run_begin(units, blocks, blockIdx.x + 1);
  const long long lo = b_lo + run_begin(b_hi - b_lo, C::WARPS, warp);
  const long long hi = b_lo + run_begin(b_hi - b_lo, C::WARPS, warp + 1);

  // A warp's part of a segment begun before its run (0), and of one that goes on behind it (1).
  auto part_at = [&](int w, int which) {
    return reinterpret_cast<float*>(which == 0 ? smem + C::WARPS * C::RINGB + w * (C::PART * 4) : smem + w * C::RINGB);
  };
  unsigned char* ring = smem + warp * C::RINGB;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  if (lo < hi) {
    // The request, segment and stage of unit lo.
    Cursor cons;
    long long seg_us;  // the consumer's segment: its first unit
    {
      int a = 0, b = NTHR;
      while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (pre[m] <= lo)
          a = m;
        else
          b = m;
      }
      long long base = pre[a];
      int i = a * per;
      for (;; ++i) {
        cons.q = load_req<C>(A, i);
        const long long n = static_cast<long long>(cons.q.segs) * cons.q.stages;
        if (lo < base + n) break;
        base += n;
      }
      cons.i = i;
      cons.seg = static_cast<int>((lo - base) / cons.q.stages);
      cons.tile = static_cast<int>((lo - base) % cons.q.stages);
      seg_us = lo - cons.tile;
    }
    Cursor prod = cons;
    long long todo = hi - lo;  // units that the producer has still to fetch pages for

    // The pages of the producer's stage, one per 16 tokens, in lanes 0 .. GROUPS - 1 (-1: none).
    auto fetch_pages = [&]() {
      int page = -1;
      const int tok = (prod.q.st0 + prod.tile) * TOK + 16 * lane;
      if (lane < C::GROUPS && tok < prod.q.end) {
        page = A.table[prod.i * A.table_stride + (tok >> A.shift)];
        if (page >= A.num_pages) page = -1;
      }
      return page;
    };
    int dst[D / 64];
#pragma unroll
    for (int it = 0; it < D / 64; ++it) dst[it] = swz<D>((it * 32 + lane) / C::CH, (it * 32 + lane) % C::CH);
    auto issue = [&](int slot, int pages) {
      const uint32_t st = ring_s + slot * C::STAGEB;
      const int tok0 = (prod.q.st0 + prod.tile) * TOK, h = prod.seg % A.Hkv;
#pragma unroll
      for (int j = 0; j < C::GROUPS; ++j) {
        const int page = __shfl_sync(0xffffffffu, pages, j);
        const int bytes = page >= 0 ? 16 : 0;
        const int64_t row = max(page, 0) * A.page_rows + (static_cast<int64_t>(h) << A.shift) +
                            ((tok0 + 16 * j) & ((1 << A.shift) - 1));
        const char* k = reinterpret_cast<const char*>(A.k_codes) + row * C::ROWB + lane * 16;
        const char* v = reinterpret_cast<const char*>(A.v_codes) + row * C::ROWB + lane * 16;
#pragma unroll
        for (int it = 0; it < D / 64; ++it) {
          cp16(st + j * C::TILEB + dst[it], k + it * 512, bytes);
          cp16(st + TOK * C::ROWB + j * C::TILEB + dst[it], v + it * 512, bytes);
        }
      }
      // params, 16 bytes a lane: lanes 0-15 the keys' (four to a group), 16-31 the values'
      const int j = (lane & 15) >> 2;
      const int page = __shfl_sync(0xffffffffu, pages, j % C::GROUPS);
      const int64_t row = max(page, 0) * A.page_rows + (static_cast<int64_t>(h) << A.shift) +
                          ((tok0 + 16 * j) & ((1 << A.shift) - 1)) + (lane & 3) * 4;
      if (j < C::GROUPS)
        cp16(st + C::PAR + (lane < 16 ? 0 : TOK * 4) + (lane & 15) * 16, (lane < 16 ? A.k_param : A.v_param) + row,
             page >= 0 ? 16 : 0);
    };

    int pages = fetch_pages();
    auto produce = [&](int slot) {
      if (todo > 0) {
        issue(slot, pages);
        --todo;
        if (todo > 0) {
          advance<C>(A, prod);
          pages = fetch_pages();
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) produce(s);

    // Per segment: q as digit fragments, per column its scale, sum and limits.
    uint32_t qb[NT][KW][3][2];
    int ci[NT][3][2];
    float qsc[NT][2], xs[NT][2], m[NT][2], l[NT][2], zs[NT][2];
    int lim_hi[NT][2], lim_lo[NT][2];
    int all_hi = 0, all_lo = 0;  // tokens in [all_lo, all_hi) are seen by every column
    float acc[MT][NT][4];
    float vscale = 0.f;  // power of two that the value scales are multiplied by
    int slot = 0;
    bool fresh = true;

    for (long long u = lo; u < hi; ++u) {
      if (fresh) {
        fresh = false;
        vscale = 0.f;
        const int h = cons.seg % A.Hkv, c0 = cons.seg / A.Hkv * C::COLS, cols = cons.q.rows * group;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int c = c0 + 8 * n + g;
          uint4 w[KW];
          const uint16_t* src = A.q + (cons.q.row0 + c / group) * A.q_stride +
                                static_cast<int64_t>(h * group + c % group) * D + 8 * KW * t;
          uint32_t big = 0;
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            w[j] = c < cols ? *reinterpret_cast<const uint4*>(src + 8 * j) : make_uint4(0, 0, 0, 0);
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[j]);
#pragma unroll
            for (int z = 0; z < 4; ++z) big = max(big, max(p[z] & 0x7FFFu, (p[z] >> 16) & 0x7FFFu));
          }
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
          const bool finite = big < 0x7F80u;
          const int e = finite ? max(static_cast<int>(big >> 7) - 127, -100) : 0;
          const float up = __int_as_float((127 + 21 - e) << 23);  // 2^(21 - e)
          int s0 = 0, s1 = 0, s2 = 0;
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[j]);
            uint32_t b[3][2] = {};
#pragma unroll
            for (int z = 0; z < 8; ++z) {  // dim 8 (KW t + j) + z
              const uint16_t bits = static_cast<uint16_t>(p[z >> 1] >> (16 * (z & 1)));
              const int X = finite ? __float2int_rn(sfd::bf16_bits_to_float(bits) * up) : 0;
              const int d0 = static_cast<int8_t>(X & 0xFF), X1 = (X - d0) >> 8;
              const int d1 = static_cast<int8_t>(X1 & 0xFF), d2 = (X1 - d1) >> 8;
              s0 += d0;
              s1 += d1;
              s2 += d2;
              b[0][z & 1] |= static_cast<uint32_t>(d0 & 0xFF) << (8 * (z >> 1));
              b[1][z & 1] |= static_cast<uint32_t>(d1 & 0xFF) << (8 * (z >> 1));
              b[2][z & 1] |= static_cast<uint32_t>(d2 & 0xFF) << (8 * (z >> 1));
            }
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              qb[n][j][z][0] = b[z][0];
              qb[n][j][z][1] = b[z][1];
            }
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            s0 += __shfl_xor_sync(0xffffffffu, s0, o);
            s1 += __shfl_xor_sync(0xffffffffu, s1, o);
            s2 += __shfl_xor_sync(0xffffffffu, s2, o);
          }
          const float sc = finite ? __int_as_float((127 - 21 + e) << 23) * A.scale * kLog2e : NAN;
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // this lane's score columns 2t, 2t + 1
            const int from = (2 * t + z) * 4;
            const int t0 = __shfl_sync(0xffffffffu, s0, from), t1 = __shfl_sync(0xffffffffu, s1, from),
                      t2 = __shfl_sync(0xffffffffu, s2, from);
            ci[n][0][z] = -8 * t0;
            ci[n][1][z] = -8 * t1;
            ci[n][2][z] = -8 * t2;
            xs[n][z] = static_cast<float>(t0 + 256 * t1 + 65536 * t2);
            qsc[n][z] = __shfl_sync(0xffffffffu, sc, from);
            const int cc = c0 + 8 * n + 2 * t + z;
            const int p = cons.q.len - (cons.q.last - (cons.q.row0 + cc / group));
            lim_hi[n][z] = cc < cols ? p + 1 : INT_MAX;
            lim_lo[n][z] = cc < cols && A.window > 0 ? p + 1 - A.window : INT_MIN;
            m[n][z] = -INFINITY;
            l[n][z] = zs[n][z] = 0.f;
          }
        }
        const int r_first = cons.q.row0 + c0 / group, r_last = cons.q.row0 + (min(c0 + C::COLS, cols) - 1) / group;
        all_hi = cons.q.len - (cons.q.last - r_first) + 1;
        all_lo = A.window > 0 ? cons.q.len - (cons.q.last - r_last) + 1 - A.window : 0;
#pragma unroll
        for (int s = 0; s < MT; ++s)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[s][n][z] = 0.f;
      }

      cp_wait<C::STAGES - 2>();
      __syncwarp();
      {
        int next = slot + C::STAGES - 1;
        if (next >= C::STAGES) next -= C::STAGES;
        produce(next);
      }
      const unsigned char* st = ring + slot * C::STAGEB;
      if (++slot == C::STAGES) slot = 0;
      const uint32_t* kpar = reinterpret_cast<const uint32_t*>(st + C::PAR);
      const uint32_t* vpar = kpar + TOK;
      const int tok0 = (cons.q.st0 + cons.tile) * TOK;
      bool odd = false;  // a token of the stage does not exist, or not every column sees every token
#pragma unroll
      for (int z = 0; z < TOK; z += 32) odd |= (kpar[z + lane] & 0xFFFFu) == 0;
      odd = __any_sync(0xffffffffu, odd) || tok0 + TOK > all_hi || tok0 < all_lo;

      // scores of rows ra, rb (tokens) x columns 2t, 2t + 1, in base 2
      const int ra = (g >> 1) + 4 * (g & 1), rb = ra + 8;
      float s[TILES][NT][4];
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        uint32_t wa[KW], wb[KW];
        const unsigned char* kt = st + j * C::TILEB;
        if constexpr (D == 64) {
          *reinterpret_cast<uint2*>(wa) = *reinterpret_cast<const uint2*>(kt + swz<D>(ra, t >> 1) + 8 * (t & 1));
          *reinterpret_cast<uint2*>(wb) = *reinterpret_cast<const uint2*>(kt + swz<D>(rb, t >> 1) + 8 * (t & 1));
        } else {
#pragma unroll
          for (int z = 0; z < KW / 4; ++z) {
            *reinterpret_cast<uint4*>(wa + 4 * z) = *reinterpret_cast<const uint4*>(kt + swz<D>(ra, KW / 4 * t + z));
            *reinterpret_cast<uint4*>(wb + 4 * z) = *reinterpret_cast<const uint4*>(kt + swz<D>(rb, KW / 4 * t + z));
          }
        }
        int d[NT][3][4];
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint32_t a0 = wa[w] & 0x0F0F0F0Fu, a1 = wb[w] & 0x0F0F0F0Fu;
          const uint32_t a2 = (wa[w] >> 4) & 0x0F0F0F0Fu, a3 = (wb[w] >> 4) & 0x0F0F0F0Fu;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int z = 0; z < 3; ++z) {
              if (w == 0)
                imma(d[n][z], a0, a1, a2, a3, qb[n][w][z][0], qb[n][w][z][1], ci[n][z][0], ci[n][z][1], ci[n][z][0],
                     ci[n][z][1]);
              else
                imma(d[n][z], a0, a1, a2, a3, qb[n][w][z][0], qb[n][w][z][1], d[n][z][0], d[n][z][1], d[n][z][2],
                     d[n][z][3]);
            }
        }
        const uint32_t pa = kpar[16 * j + ra], pb = kpar[16 * j + rb];
        const float sa = sfd::half_bits_to_float(pa & 0xFFFF), za = sfd::half_bits_to_float(pa >> 16) - 8.f;
        const float sb = sfd::half_bits_to_float(pb & 0xFFFF), zb = sfd::half_bits_to_float(pb >> 16) - 8.f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float f = fmaf(static_cast<float>(d[n][2][z] * 256 + d[n][1][z]), 256.f,
                                 static_cast<float>(d[n][0][z]));
            s[j][n][z] = fmaf(z < 2 ? -za : -zb, xs[n][z & 1], f) * ((z < 2 ? sa : sb) * qsc[n][z & 1]);
          }
        if (odd) {
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const int tok = tok0 + 16 * j + (z < 2 ? ra : rb);
            const bool there = ((z < 2 ? pa : pb) & 0xFFFFu) != 0;
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (!there || tok >= lim_hi[n][z & 1] || tok < lim_lo[n][z & 1]) s[j][n][z] = -INFINITY;
          }
        }
      }

      // the stage's value scales and zero points
      float vs[TILES][2], vz[TILES][2], vmax = 0.f;
#pragma unroll
      for (int j = 0; j < TILES; ++j)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          uint32_t p = vpar[16 * j + (z ? rb : ra)];
          // a token that no column sees may hold anything: its weight 0 must stay 0
          if (odd && ((p & 0x7C00u) == 0x7C00u || (p & 0x7C000000u) == 0x7C000000u)) p = 0;
          vs[j][z] = sfd::half_bits_to_float(p & 0xFFFF);
          vz[j][z] = sfd::half_bits_to_float(p >> 16) - 8.f;
          vmax = fmaxf(vmax, fabsf(vs[j][z]));
        }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
      float grow = 1.f;
      if (vmax * vscale >= 2048.f || (vscale == 0.f && vmax > 0.f)) {
        // 2^(10 - exponent of vmax), exact
        const float next = __int_as_float((127 + 10 + 127 - (__float_as_int(vmax) >> 23)) << 23);
        if (vscale != 0.f) grow = next / vscale;
        vscale = next;
      }

      // running maxima and the rescaling of what has been summed
      bool rescale = grow != 1.f;
      float alpha[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float mx = m[n][z];
#pragma unroll
          for (int j = 0; j < TILES; ++j) mx = fmaxf(mx, fmaxf(s[j][n][z], s[j][n][z + 2]));
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float use = mx == -INFINITY ? 0.f : mx;
          alpha[n][z] = ex2(m[n][z] - use);
          rescale |= mx != m[n][z];
          m[n][z] = mx;
#pragma unroll
          for (int j = 0; j < TILES; ++j) {
            s[j][n][z] = ex2(s[j][n][z] - use);
            s[j][n][z + 2] = ex2(s[j][n][z + 2] - use);
          }
        }
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            l[n][z] *= alpha[n][z];
            alpha[n][z] *= grow;
            zs[n][z] *= alpha[n][z];
          }
#pragma unroll
          for (int k = 0; k < MT; ++k)
#pragma unroll
            for (int z = 0; z < 4; ++z) acc[k][n][z] *= alpha[n][z & 1];
        }
      }

      // values
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // row ra, row rb
            const float p0 = s[j][n][2 * z], p1 = s[j][n][2 * z + 1], sc = vs[j][z] * vscale;
            l[n][0] += p0;
            l[n][1] += p1;
            const float w0 = p0 * sc, w1 = p1 * sc;
            zs[n][0] = fmaf(w0, vz[j][z], zs[n][0]);
            zs[n][1] = fmaf(w1, vz[j][z], zs[n][1]);
            const __half2 hi2 = __floats2half2_rn(w0, w1);
            const float2 back = __half22float2(hi2);
            const __half2 lo2 = __floats2half2_rn(w0 - back.x, w1 - back.y);
            bh[n][z] = transpose8x8(reinterpret_cast<const uint32_t&>(hi2));
            bl[n][z] = transpose8x8(reinterpret_cast<const uint32_t&>(lo2));
          }
        uint32_t v[4][VW];  // tokens t, t + 4, t + 8, t + 12
        const unsigned char* vt = st + TOK * C::ROWB + j * C::TILEB;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const int r = t + 4 * z;
          if constexpr (D == 64)
            v[z][0] = *reinterpret_cast<const uint32_t*>(vt + swz<D>(r, g >> 2) + 4 * (g & 3));
          else if constexpr (D == 128)
            *reinterpret_cast<uint2*>(v[z]) = *reinterpret_cast<const uint2*>(vt + swz<D>(r, g >> 1) + 8 * (g & 1));
          else
            *reinterpret_cast<uint4*>(v[z]) = *reinterpret_cast<const uint4*>(vt + swz<D>(r, g));
        }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t x0 = __byte_perm(v[0][w], v[1][w], b | (4 + b) << 8 | b << 4 | (4 + b) << 12);
            const uint32_t x1 = __byte_perm(v[2][w], v[3][w], b | (4 + b) << 8 | b << 4 | (4 + b) << 12);
            const uint32_t a0 = nib_lo(x0), a1 = nib_hi(x0), a2 = nib_lo(x1), a3 = nib_hi(x1);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              hmma(acc[4 * w + b][n], a0, a1, a2, a3, bh[n][0], bh[n][1]);
              hmma(acc[4 * w + b][n], a0, a1, a2, a3, bl[n][0], bl[n][1]);
            }
          }
      }

      // the segment's end, or the run's
      const bool seg_done = cons.tile + 1 == cons.q.stages;
      if (seg_done || u + 1 == hi) {
        const long long seg_ue = seg_us + cons.q.stages;
        const bool whole = seg_us >= lo && seg_ue <= hi;
        const int which = seg_us < lo ? 0 : 1;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              l[n][z] += __shfl_xor_sync(0xffffffffu, l[n][z], o);
              zs[n][z] += __shfl_xor_sync(0xffffffffu, zs[n][z], o);
            }
            const float inv = l[n][z] == 0.f ? 0.f : 1.f / (l[n][z] * (vscale == 0.f ? 1.f : vscale));
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              acc[k][n][z] = (acc[k][n][z] - zs[n][z]) * inv;
              acc[k][n][z + 2] = (acc[k][n][z + 2] - zs[n][z]) * inv;
            }
          }
        if (whole) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
              for (int k = 0; k < MT; ++k)
                put<C>(A, cons.q, cons.seg, 8 * n + 2 * t + z, D / 8 * g + 2 * k, acc[k][n][z], acc[k][n][z + 2]);
        } else {
          // Part 1 ends the run, so it takes the drained ring's place.
          __syncwarp();
          float* keep = part_at(warp, which);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int col = 8 * n + 2 * t + z;
#pragma unroll
              for (int k = 0; k < MT; ++k)
                *reinterpret_cast<float2*>(keep + col * D + D / 8 * g + 2 * k) =
                    make_float2(acc[k][n][z], acc[k][n][z + 2]);
              if (g == 0) keep[C::COLS * D + col] = l[n][z] == 0.f ? -INFINITY : m[n][z] + log2f(l[n][z]);
            }
          if (lane == 0) parts[warp][which] = Part{seg_us, seg_ue, cons.i, cons.seg};
        }
        fresh = true;
        seg_us = u + 1;
      }
      if (u + 1 < hi) advance<C>(A, cons);
    }
  }

  // Segments that are split over the block's warps: the one begun in an earlier block, if any, then those begun in
  // each warp's run.
  __syncthreads();
  bool open = false;
  for (int s = 0; s <= C::WARPS; ++s) {
    Part p = {-1, 0, 0, 0};
    if (s == 0) {
      for (int w = 0; w < C::WARPS; ++w)
        if (parts[w][0].us >= 0 && parts[w][0].us < b_lo) p = parts[w][0];
    } else {
      p = parts[s - 1][1];
    }
    if (p.us < 0) continue;  // the same for the whole block
    const bool early = p.us < b_lo, late = p.ue > b_hi;
    const Req q = load_req<C>(A, p.i);
    for (int x = tid; x < C::COLS * (D / 4); x += NTHR) {
      const int col = x / (D / 4), dim = x % (D / 4) * 4;
      float top = -INFINITY;
      for (int w = 0; w < C::WARPS; ++w)
#pragma unroll
        for (int z = 0; z < 2; ++z)
          if (parts[w][z].us == p.us) {
            const float v = part_at(w, z)[C::COLS * D + col];
            top = v > top || v != v ? v : top;  // a NaN stays
          }
      float sum = 0.f, o[4] = {};
      for (int w = 0; w < C::WARPS; ++w)
#pragma unroll
        for (int z = 0; z < 2; ++z)
          if (parts[w][z].us == p.us) {
            const float* from = part_at(w, z);
            const float f = top == -INFINITY ? 0.f : ex2(from[C::COLS * D + col] - top);
            const float4 v = *reinterpret_cast<const float4*>(from + col * D + dim);
            sum += f;
            o[0] = fmaf(f, v.x, o[0]);
            o[1] = fmaf(f, v.y, o[1]);
            o[2] = fmaf(f, v.z, o[2]);
            o[3] = fmaf(f, v.w, o[3]);
          }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] *= inv;
      if (!early && !late) {
        put<C>(A, q, p.seg, col, dim, o[0], o[1]);
        put<C>(A, q, p.seg, col, dim + 2, o[2], o[3]);
      } else {
        float* to = W.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (early ? 0 : 1)) * C::PART;
        *reinterpret_cast<float4*>(to + col * D + dim) = make_float4(o[0], o[1], o[2], o[3]);
        if (dim == 0) to[C::COLS * D + col] = sum == 0.f ? -INFINITY : top + log2f(sum);
      }
    }
    if (!early && late) {
      open = true;
      if (tid == 0) W.tails[blockIdx.x] = Tail{1, p.i, p.seg, run_of(units, blocks, p.ue - 1)};
    }
  }
  if (!open && tid == 0) W.tails[blockIdx.x].open = 0;
}

// Joins the parts of the segment that starts in block b and ends in a later one.
template <class C>
__global__ void __launch_bounds__(256) attn_paged_join_kernel(const __grid_constant__ Work W) {
  constexpr int D = C::D;
  const Tail tail = W.tails[blockIdx.x];
  if (!tail.open) return;
  const int b = blockIdx.x, n = tail.last_cta - b + 1;
  const Req q = load_req<C>(W.a, tail.i);
  auto part = [&](int k) { return W.parts + (static_cast<int64_t>(b + k) * 2 + (k == 0 ? 1 : 0)) * C::PART; };
  for (int x = threadIdx.x; x < C::COLS * (D / 4); x += 256) {
    const int col = x / (D / 4), dim = x % (D / 4) * 4;
    float top = -INFINITY;
    for (int k = 0; k < n; ++k) {
      const float v = part(k)[C::COLS * D + col];
      top = v > top || v != v ? v : top;
    }
    float sum = 0.f, o[4] = {};
    for (int k = 0; k < n; ++k) {
      const float f = top == -INFINITY ? 0.f : ex2(part(k)[C::COLS * D + col] - top);
      const float4 v = *reinterpret_cast<const float4*>(part(k) + col * D + dim);
      sum += f;
      o[0] = fmaf(f, v.x, o[0]);
      o[1] = fmaf(f, v.y, o[1]);
      o[2] = fmaf(f, v.z, o[2]);
      o[3] = fmaf(f, v.w, o[3]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    put<C>(W.a, q, tail.seg, col, dim, o[0] * inv, o[1] * inv);
    put<C>(W.a, q, tail.seg, col, dim + 2, o[2] * inv, o[3] * inv);
  }
}

template <class C>
sf_status launch(const AttnArgs& A, void* ws, int blocks, cudaStream_t s) {
  Work W{};
  W.a = A;
  W.tails = static_cast<Tail*>(ws);
  W.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + (blocks * sizeof(Tail) + 255) / 256 * 256);
  W.blocks = blocks;
  SF_CHECK_CUDA(cudaFuncSetAttribute(attn_paged_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM));
  attn_paged_kernel<C><<<blocks, 32 * C::WARPS, C::SMEM, s>>>(W);
  sf_status st = sf::check_launch("attn_paged_kernel");
  if (st != SF_OK) return st;
  attn_paged_join_kernel<C><<<blocks, 256, 0, s>>>(W);
  return sf::check_launch("attn_paged_join_kernel");
}

using Cfg64x8 = Cfg<64, 1, 64, 8, 3>;
using Cfg64x16 = Cfg<64, 2, 64, 8, 3>;
using Cfg128x8 = Cfg<128, 1, 64, 8, 2>;
using Cfg128x16 = Cfg<128, 2, 64, 8, 2>;
using Cfg256x8 = Cfg<256, 1, 32, 8, 2>;

// Columns of a block: 16 when a request's rows can fill more than 8 (d = 256: always 8, its registers hold no more).
int block_cols(int T, int R, int Hq, int Hkv, int d) {
  const int64_t rows = (static_cast<int64_t>(T) + R - 1) / R;
  return d < 256 && rows * (Hq / Hkv) > 8 ? 16 : 8;
}

}  // namespace

extern "C" sf_status sf_attn_paged_workspace_size(int T, int R, int Hq, int Hkv, int d, size_t* bytes) {
  const char* what = "sf_attn_paged_workspace_size";
  SF_REQUIRE(bytes, "%s: null pointer", what);
  SF_REQUIRE(d == 64 || d == 128 || d == 256, "%s: d must be 64, 128 or 256", what);
  SF_REQUIRE(Hkv >= 1 && Hkv <= 256 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 64,
             "%s: need Hkv in [1, 256] and Hq/Hkv a whole number up to 64", what);
  SF_REQUIRE(T >= 0 && R >= 1 && R <= 8192, "%s: need T >= 0 and R in [1, 8192]", what);
  const size_t blocks = sf::sm_count();
  const size_t part = static_cast<size_t>(block_cols(T, R, Hq, Hkv, d)) * (d + 1) * sizeof(float);
  *bytes = (blocks * sizeof(Tail) + 255) / 256 * 256 + blocks * 2 * part;
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
  cudaStream_t s = sf::as_cuda(stream);
  const int blocks = sf::sm_count();
  if (kv.d == 256) return launch<Cfg256x8>(A, a->workspace, blocks, s);
  const bool wide = block_cols(a->T, a->R, a->Hq, kv.Hkv, kv.d) == 16;
  if (kv.d == 64)
    return wide ? launch<Cfg64x16>(A, a->workspace, blocks, s) : launch<Cfg64x8>(A, a->workspace, blocks, s);
  return wide ? launch<Cfg128x16>(A, a->workspace, blocks, s) : launch<Cfg128x8>(A, a->workspace, blocks, s);
}
