// sf_attn_paged: attention of a step's rows over a paged 4-bit KV cache.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

#include "launch.cuh"
#include "paged.cuh"

namespace {

struct AttnArgs {
  const uint32_t *k_codes, *k_param, *v_codes, *v_param;
  const uint16_t* q;
  const int32_t *cu_rows, *len, *table;
  void* out;
  int64_t q_stride, out_stride, table_stride, page_rows;
  float scale;
  int T, R, Hq, Hkv, group, shift, num_pages, max_pages, window, bf16_out;
  uint32_t per_group;  // ceil(2^32 / group): columns are below 2^26, so its high product is the quotient; 0 for 1
};

// How the work is laid out.  A request's rows times the query heads of one KV
// head are the columns that read the same keys; a column block takes COLS = 8
// NT of them.  A segment is one (request, column block, KV head); its tokens
// come in stages of TOK.  Stages of all segments, in order, are the units,
// and every block (and in it every warp) takes an equal run of them, so a
// 128K-token request and a hundred short ones fill the SMs alike.  A segment
// that lies within one warp's run is written by it; the parts of one that does
// not are joined in shared memory, and across blocks by a second kernel (the last
// block to arrive doing it instead was slower: two fences, and the same reads).
//
// A warp's stage of 16-token tiles:
//  * scores: mma.m16n8k32 (s8), rows = tokens, columns = query columns.  A
//    4-bit code word is two operand registers by two masks, even codes as c, odd
//    ones as 16 c, kept in sums of their own (16 columns: the odd ones shifted
//    instead, which costs less than twice the sums).  q enters as
//    X = rint(q 2^(21-e)) (e the exponent of its row's largest entry) in three
//    balanced base-256 digits, one product each: exact in 32-bit integers, and
//    half the instructions of f16 codes.  The zero point takes z sum X off;
//  * softmax in base 2 against a reference per column, put 2 above the largest
//    score and raised only when one exceeds it by 4, so most steps need a vote,
//    not a reduction;
//  * values: mma.m16n8k16 (f16), rows = dims, columns = query columns, k =
//    tokens.  A byte permute pairs the codes of two tokens, a mask-and-or makes
//    them 1024 + c (bits 0-3) or 1024 + 16 c (bits 4-7), one exact f16 operation
//    on the FMA pipe c - 8.  (Taken as f16 subnormals, c 2^-24 and c 2^-20, they
//    need masks only, but a product's low bits are then cut off: 4e-4 at 128K
//    tokens.)  The weights p v_s enter as an f16 value and
//    its f16 remainder (22 bits; v_s scaled by a power of two that follows the
//    largest seen); movmatrix turns them from score order to operand order.  The
//    tensor cores truncate their fp32 sums, so a chain of them drifts (7e-6 over
//    a run of 112): after FLUSH stages the sums are added, rounded, to sums in
//    shared memory and start again (128K tokens: 0.8e-6 off with a flush every 64
//    tokens; every 256 in 2% less time, 1.4e-6; none in 4% less, 4.4e-6; sums in
//    the workspace instead cost 20%);
//  * PACK, up to 4 columns (a decode step with 4 query heads per KV head): the
//    score products' 16 columns are digit 0, digit 1 and twice digit 2 of the
//    four, so a lane keeps one of its two tokens and half the softmax work, and
//    the value product's columns are the four weights and their four remainders:
//    half the products.
// The output's type decides nothing but the last rounding.  (Two digits of q and
// weights without remainders for bf16 outputs take 23% less time, 185 us for 241
// with 64 requests of 1 to 4 rows, but lose bits of every channel below a
// query's largest, and show in the bf16 output.)
// The k index of the value product is free, so the tokens of a tile are
// ordered such that both fragment loads are free of bank conflicts.
//
// The cache streams through a ring of STAGES stages per warp (cp.async, no
// barrier between warps), across segment ends, the block table's entries a
// stage ahead of that.

// log2(e)
constexpr float kLog2e = 1.4426950408889634f;

template <int D_, int NT_, bool PACK_, int TOK_, int WARPS_, int STAGES_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, TOK = TOK_, WARPS = WARPS_, STAGES = STAGES_;
  static constexpr bool PACK = PACK_;
  static constexpr int FLUSH = 64 / TOK;  // stages
  static constexpr int COLS = PACK ? 4 : 8 * NT, GROUPS = TOK / 16;
  // tiles and tokens of a step of the inner loop: four tiles where the registers allow (128K tokens: 44 us; two, 47)
  static constexpr int TILES = NT == 1 && D <= 128 && WARPS == 8 ? 4 : 2, SUB = 16 * TILES;
  static_assert(TOK % SUB == 0, "whole steps");
  static constexpr bool SPLIT = NT == 1;  // odd codes as 16 c in sums of their own: fewer shifts, more sums
  static constexpr int DT = PACK ? 2 : 3;                      // products of 8 columns per k step and column tile
  static constexpr int ROWS = PACK ? 1 : 2;                    // tokens of a tile whose scores a lane keeps
  static constexpr int KW = D / 32, VW = D / 64, MT = D / 16;  // words per lane of a K row, of a V row; dim tiles
  static constexpr int ROWB = D / 2, TILEB = 16 * ROWB, CH = D / 32;  // bytes of a row and of a tile; 16-byte chunks
  static constexpr int PAR = 2 * TOK * ROWB;                          // offset of the params in a stage
  static constexpr int STAGEB = PAR + 2 * TOK * 4;
  static constexpr int PART = COLS * (D + 1);  // floats of one partial: the columns' outputs, then their log sums
  static constexpr int JOIN = COLS == 4 ? 4 : 2;  // warps a column of the second kernel
  static constexpr int SUMS = MT * NT * 4 * 32;  // a warp's value sums
  static constexpr int RINGB = STAGES * STAGEB;
  static constexpr int SMEM = WARPS * (RINGB + SUMS * 4);  // the rings, then each warp's flushed sums
  static_assert(!PACK || NT == 1, "packed columns are one tile");
  static_assert(PART * 4 <= RINGB, "a warp's partial takes its ring's place");
  static_assert(SMEM <= 224 * 1024, "shared memory");
};

// Offset in a 16-token tile of chunk ch (16 bytes) of row r: rows k and k + 4
// (a K load's quarter warp) and rows 4j .. 4j + 3 (a V load's) meet no bank
// twice.  Row r + 8 is always 8 ROWB behind row r.
template <int D>
__device__ __forceinline__ int swz(int r, int ch) {
  if constexpr (D == 64) return ((r & ~3) | ((r & 3) ^ (2 * ((r >> 2) & 1)))) * 32 + ch * 16;
  if constexpr (D == 128)
    return (r >> 1) * 128 + (((r & 1) ^ ((r >> 2) & 1)) * 64) + ((ch ^ (2 * ((r >> 1) & 1))) * 16);
  return r * 128 + ((ch ^ ((2 * (r & 3)) | ((r >> 2) & 1))) * 16);
}

// 16 bytes from src + SRC to dst + DST; _if: zeros where there is nothing to copy.
template <int DST, int SRC>
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;\n" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC));
}
template <int DST, int SRC>
__device__ __forceinline__ void cp16_if(uint32_t dst, const void* src, bool there) {
  asm volatile(
      "{ .reg .pred none; setp.eq.s32 none, %2, 0; cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, none; }\n" ::"r"(
          dst),
      "l"(src), "r"(static_cast<int>(there)), "n"(DST), "n"(SRC));
}
// A tile's codes, for copies Z .. : copy 2 it goes to d0, 2 it + 1 to d1 (d = 256), all to d0 (else).
template <class C, int SRC0, int DST0, int IT = 0>
__device__ __forceinline__ void cp_tile(uint32_t d0, uint32_t d1, const char* src) {
  constexpr int kDst = DST0 + (C::D == 256 ? (IT >> 1) * 8 * C::ROWB : IT * 512);
  cp16<kDst, SRC0 + IT * 512>(C::D == 256 && (IT & 1) ? d1 : d0, src);
  if constexpr (IT + 1 < C::D / 64) cp_tile<C, SRC0, DST0, IT + 1>(d0, d1, src);
}
template <class C, int DST0, int IT = 0>
__device__ __forceinline__ void cp_tile_if(uint32_t d0, uint32_t d1, const char* src, bool there) {
  constexpr int kDst = DST0 + (C::D == 256 ? (IT >> 1) * 8 * C::ROWB : IT * 512);
  cp16_if<kDst, IT * 512>(C::D == 256 && (IT & 1) ? d1 : d0, src, there);
  if constexpr (IT + 1 < C::D / 64) cp_tile_if<C, DST0, IT + 1>(d0, d1, src, there);
}
// Tiles J .. of a stage that lies in one page.
template <class C, int J = 0>
__device__ __forceinline__ void cp_stage(uint32_t d0, uint32_t d1, const char* k, const char* v) {
  cp_tile<C, J * C::TILEB, J * C::TILEB>(d0, d1, k);
  cp_tile<C, J * C::TILEB, C::TOK * C::ROWB + J * C::TILEB>(d0, d1, v);
  if constexpr (J + 1 < C::GROUPS) cp_stage<C, J + 1>(d0, d1, k, v);
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
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// The nibbles at bits 0-3 and 16-19 (lo), 4-7 and 20-23 (hi) of x as f16 c - 8.
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(mask), "r"(bits));  // (x & mask) | bits
  return y;
}
__device__ __forceinline__ uint32_t nib_lo(uint32_t x) {
  const uint32_t v = and_or(x, 0x000F000Fu, 0x64006400u);  // 1024 + c
  const __half2 r = __hsub2(reinterpret_cast<const __half2&>(v), __float2half2_rn(1032.f));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t nib_hi(uint32_t x) {
  const uint32_t v = and_or(x, 0x00F000F0u, 0x64006400u);  // 1024 + 16 c
  const __half2 r =
      __hfma2(reinterpret_cast<const __half2&>(v), __float2half2_rn(0.0625f), __float2half2_rn(-72.f));
  return reinterpret_cast<const uint32_t&>(r);
}

__device__ __forceinline__ uint32_t h2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return reinterpret_cast<const uint32_t&>(h);
}

// Column c's row: c / group.
__device__ __forceinline__ int row_of(const AttnArgs& A, int c) {
  return A.per_group == 0 ? c : static_cast<int>(__umulhi(static_cast<uint32_t>(c), A.per_group));
}

// The first token that the row at position p sees; p may be negative, and the window as long as an int can say.
__device__ __forceinline__ int window_begin(const AttnArgs& A, int p) {
  return A.window > 0 && p >= A.window ? p - A.window + 1 : 0;
}

// One request's columns and stages.
struct Req {
  int row0, rows;    // its rows in q and out (those below T)
  int last;          // cu_rows[i + 1]: row t is the token at len - (last - t)
  int len, end;      // tokens held; tokens that its last row sees
  int st0, stages;   // first stage, number of stages (at least 1)
  int blocks;        // column blocks: blocks Hkv segments, the KV head fastest
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
  q.st0 = window_begin(A, first) / C::TOK;
  q.stages = max((q.end - 1) / C::TOK + 1 - q.st0, 1);
  q.blocks = (q.rows * A.group + C::COLS - 1) / C::COLS;
  return q;
}

// A place in the run of units.
struct Cursor {
  Req q;
  int i, block, h, tile;
};

template <class C>
__device__ __forceinline__ void advance(const AttnArgs& A, Cursor& c) {
  if (++c.tile < c.q.stages) return;
  c.tile = 0;
  if (++c.h < A.Hkv) return;
  c.h = 0;
  if (++c.block < c.q.blocks) return;
  c.block = 0;
  do {
    ++c.i;
    if (c.i >= A.R) return;
    c.q = load_req<C>(A, c.i);
  } while (c.q.blocks == 0);
}

// What the second kernel needs of a block: the segment that starts in it and
// ends in a later block.
struct Tail {
  int open;         // 1: there is one
  int row0, rows;   // its request's
  int block, h;     // which of the request's
  int last_cta;     // the block that holds its last unit
};

struct Work {
  AttnArgs a;
  Tail* tails;    // [blocks]
  float* parts;   // [blocks][2][PART]: a block's part of a segment begun earlier (0), of its open one (1)
  float* heads;   // [blocks][WARPS][PART]: a warp's part of a segment begun before its run, when the run goes on
  int blocks;
};

// a / b for a >= 0, b > 0, in 32 bits where they do.
__device__ __forceinline__ long long quot(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// n equal runs of u units: each has `size`, the first `more` of them one more.
struct Runs {
  long long size;
  int more;
  __device__ Runs(long long u, int n) : size(quot(u, n)), more(static_cast<int>(u - size * n)) {}
  __device__ long long begin(int c) const { return size * c + min(c, more); }
  __device__ int of(long long x) const {  // the run that holds unit x
    const long long big = (size + 1) * more;
    return static_cast<int>(x < big ? quot(x, size + 1) : more + quot(x - big, size));
  }
};

// Dims x .. x + 3 of a column of a segment.
template <class C>
__device__ __forceinline__ void put(const AttnArgs& A, int row0, int rows, int block, int h, int col, int x, float4 v) {
  const int c = block * C::COLS + col;
  if (c >= rows * A.group) return;
  const int r = row_of(A, c);
  const int64_t at = (row0 + r) * A.out_stride + static_cast<int64_t>(h * A.group + c - r * A.group) * C::D + x;
  if (A.bf16_out) {
    __nv_bfloat162 b[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(A.out) + at) = *reinterpret_cast<const uint2*>(b);
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(A.out) + at) = v;
  }
}

// The warp joins column col of n <= 32 parts (lane k < n: part k's address) and hands dims and log sum on: lane l gets
// dims 4 l + 128 k.  lse: the lane's part's log sum (-inf beyond n), top: the largest of all.  In the parts' order.
template <class C>
__device__ __forceinline__ void join_column(const float* at, int n, int col, float lse, float top, float& sum,
                                            float4 (&o)[(C::D + 127) / 128]) {
  constexpr int D = C::D;
  const int lane = threadIdx.x & 31;
  const float f = top != -INFINITY ? ex2(lse - top) : 0.f;
  const unsigned long long mine = reinterpret_cast<unsigned long long>(at);
#pragma unroll 8
  for (int k = 0; k < n; ++k) {
    const float* from = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, mine, k)) + col * D + 4 * lane;
    const float w = __shfl_sync(0xffffffffu, f, k);
    sum += w;
#pragma unroll
    for (int z = 0; z < (D + 127) / 128; ++z) {
      if (D < 128 && 4 * lane >= D) continue;
      const float4 v = *reinterpret_cast<const float4*>(from + 128 * z);
      o[z].x = fmaf(w, v.x, o[z].x);
      o[z].y = fmaf(w, v.y, o[z].y);
      o[z].z = fmaf(w, v.z, o[z].z);
      o[z].w = fmaf(w, v.w, o[z].w);
    }
  }
}

// Maximum over the warp that a NaN wins.
__device__ __forceinline__ float warp_top(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, v, o);
    v = v != v || v > y ? v : y;
  }
  return v;
}

template <class C>
__global__ void __launch_bounds__(32 * C::WARPS, 1) attn_paged_kernel(const __grid_constant__ Work W) {
  constexpr int D = C::D, NT = C::NT, TOK = C::TOK, TILES = C::TILES, KW = C::KW, VW = C::VW, MT = C::MT;
  constexpr int ROWS = C::ROWS, NTHR = 32 * C::WARPS;
  constexpr bool PACK = C::PACK;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long pre[NTHR + 1];  // units before each thread's run of requests
  __shared__ long long wsum[C::WARPS];
  struct Part {
    long long us, ue;  // the segment's units; us < 0: none
    const float* at;
    int row0, rows, block, h;
  };
  __shared__ Part parts[C::WARPS][2];  // of the segment begun before the warp's run, and of the one that goes on behind
  const AttnArgs& A = W.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int group = A.group;

  sfd::wait_for_previous();
  sfd::let_next_prepare();

  // The units of all requests.
  const int per = (A.R + NTHR - 1) / NTHR;
  long long mine = 0;
  for (int i = min(tid * per, A.R); i < min((tid + 1) * per, A.R); ++i) {
    const Req q = load_req<C>(A, i);
    mine += static_cast<long long>(q.blocks) * A.Hkv * q.stages;
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
    if (tid == 0) W.tails[blockIdx.x].open = 0;
    return;
  }
  const Runs runs(units, blocks);
  const long long b_lo = runs.begin(blockIdx.x), b_hi = runs.begin(blockIdx.x + 1);
  const int b_units = static_cast<int>(b_hi - b_lo), w_size = b_units / C::WARPS, w_more = b_units % C::WARPS;
  const long long lo = b_lo + w_size * warp + min(warp, w_more);
  const int count = w_size + (warp < w_more);

  unsigned char* ring = smem + warp * C::RINGB;
  const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  if (count > 0) {
    // The request, segment and stage of unit lo.
    Cursor cons;
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
        const long long n = static_cast<long long>(cons.q.blocks) * A.Hkv * cons.q.stages;
        if (lo < base + n) break;
        base += n;
      }
      const int seg = static_cast<int>(quot(lo - base, cons.q.stages));
      cons.i = i;
      cons.tile = static_cast<int>((lo - base) - static_cast<long long>(seg) * cons.q.stages);
      cons.block = seg / A.Hkv;
      cons.h = seg - cons.block * A.Hkv;
    }
    Cursor prod = cons;
    int todo = count;             // units that the producer has still to issue
    int seg_at = -cons.tile;      // the consumer's segment: its first unit, counted from lo

    // The first rows of the producer's stage in the pool, one per 16 tokens, in lanes 0 .. GROUPS - 1 (-1: no page).
    auto fetch_rows = [&]() {
      long long row = -1;
      const int tok = (prod.q.st0 + prod.tile) * TOK + 16 * lane;
      if (lane < C::GROUPS && tok < prod.q.end) {
        const int page = A.table[prod.i * A.table_stride + (tok >> A.shift)];
        if (page >= 0 && page < A.num_pages)
          row = static_cast<long long>(page) * A.page_rows +
                ((prod.h << A.shift) + (tok & ((1 << A.shift) - 1)));
      }
      return row;
    };
    // where the lane's chunks of a tile go (cp_tile: 512 bytes on in the pool is 512/ROWB rows on)
    const uint32_t dst0 = ring_s + swz<D>(lane / C::CH, lane % C::CH);
    const uint32_t dst1 = ring_s + swz<D>(lane / C::CH + 4, lane % C::CH);
    const char* const k_lane = reinterpret_cast<const char*>(A.k_codes) + lane * 16;
    const char* const v_lane = reinterpret_cast<const char*>(A.v_codes) + lane * 16;
    // params, 16 bytes a lane: lanes 0-15 the keys' (four to a group), 16-31 the values'
    const char* const p_lane = reinterpret_cast<const char*>(lane < 16 ? A.k_param : A.v_param) + (lane & 3) * 16;
    const int p_group = (lane & 15) >> 2;
    const uint32_t p_dst = ring_s + C::PAR + (lane < 16 ? 0 : TOK * 4) + (lane & 15) * 16;
    auto issue = [&](int slot, long long rows) {
      const uint32_t st = slot * C::STAGEB;
      const long long r0 = __shfl_sync(0xffffffffu, rows, 0);
      if ((1 << A.shift) >= TOK && r0 >= 0) {  // the stage lies in one page
        cp_stage<C>(dst0 + st, dst1 + st, k_lane + r0 * C::ROWB, v_lane + r0 * C::ROWB);
        if (p_group < C::GROUPS) cp16<0, 0>(p_dst + st, p_lane + r0 * 4 + p_group * 64);
        return;
      }
#pragma unroll
      for (int j = 0; j < C::GROUPS; ++j) {
        const long long r = __shfl_sync(0xffffffffu, rows, j), at = max(r, 0ll) * C::ROWB;
        cp_tile_if<C, 0>(dst0 + st + j * C::TILEB, dst1 + st + j * C::TILEB, k_lane + at, r >= 0);
        cp_tile_if<C, TOK * C::ROWB>(dst0 + st + j * C::TILEB, dst1 + st + j * C::TILEB, v_lane + at, r >= 0);
      }
      const long long r = __shfl_sync(0xffffffffu, rows, p_group % C::GROUPS);
      if (p_group < C::GROUPS) cp16_if<0, 0>(p_dst + st, p_lane + max(r, 0ll) * 4, r >= 0);
    };
    long long rows = fetch_rows();
    auto produce = [&](int slot) {
      if (todo > 0) {
        issue(slot, rows);
        if (--todo > 0) {
          advance<C>(A, prod);
          rows = fetch_rows();
        }
      }
      cp_commit();
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) produce(s);

    // Per segment: q as operand fragments; per column its score scale, sum of q and limits.
    uint32_t qb[NT][KW / 2][C::DT][2][2];  // [word pair][digits][the pair's products][operand registers]
    auto b_at = [&](int n, int word, int y, int odd) -> uint32_t& {
      return C::SPLIT ? qb[n][word / 2][y][odd][word & 1] : qb[n][word / 2][y][word & 1][odd];
    };
    float qsc[NT][2], qsum[NT][2], m[NT][2], l[NT][2], zs[NT][2];
    int lim_hi[NT][2], lim_lo[NT][2];
    int all_hi = 0, all_lo = 0;  // tokens in [all_lo, all_hi) are seen by every column
    int any_hi = 0, any_lo = 0;  // those outside [any_lo, any_hi) by none
    float acc[MT][NT][4];  // the value sums since the last flush
    float4* const flushed = reinterpret_cast<float4*>(smem + C::WARPS * C::RINGB) + warp * (C::SUMS / 4) + lane;
    int since = 0;         // stages in acc
    bool has_flushed = false, empty = true;  // empty: nothing in acc yet
    float vscale = 0.f;  // power of two that the value scales are multiplied by
    int slot = 0;
    bool fresh = true;
    // the lane's score columns within a tile of 8, and its tokens within a tile of 16
    const int col0 = PACK ? 2 * (t & 1) : 2 * t;
    const int ra = (g >> 1) + 4 * (g & 1), rb = ra + 8;
    const int tok_of[2] = {PACK && t >= 2 ? rb : ra, rb};
    const float own_w = t < 2 ? 1.f : 256.f, other_w = t < 2 ? 256.f : 1.f;  // packed: the weights of digits 0 and 1
    // its words of a K row (row ra; rb is 8 rows on) and of V rows t, t + 4 (t + 8 and t + 12 are 8 rows on)
    const int k_off = D == 64 ? swz<D>(ra, t >> 1) + 8 * (t & 1) : swz<D>(ra, KW / 4 * t);
    const int k_off1 = D == 256 ? swz<D>(ra, 2 * t + 1) : 0;
    auto v_at = [&](int r) {
      return TOK * C::ROWB + (D == 64    ? swz<D>(r, g >> 2) + 4 * (g & 3)
                              : D == 128 ? swz<D>(r, g >> 1) + 8 * (g & 1)
                                         : swz<D>(r, g));
    };
    const int v_off0 = v_at(t), v_off1 = v_at(t + 4);

    for (int u = 0; u < count; ++u) {
      if (fresh) {
        fresh = false;
        empty = true;
        vscale = 0.f;
        const int h = cons.h, c0 = cons.block * C::COLS, cols = cons.q.rows * group;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int c = c0 + (PACK ? g & 3 : 8 * n + g);
          uint4 w[KW];
          const int r = row_of(A, c);
          const uint16_t* src = A.q + (cons.q.row0 + r) * A.q_stride +
                                static_cast<int64_t>(h * group + c - r * group) * D + 8 * KW * t;
          uint32_t big = 0;  // two halves
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            w[j] = c < cols ? *reinterpret_cast<const uint4*>(src + 8 * j) : make_uint4(0, 0, 0, 0);
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[j]);
#pragma unroll
            for (int z = 0; z < 4; ++z) big = __vmaxu2(big, p[z] & 0x7FFF7FFFu);
          }
          big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 1));
          big = __vmaxu2(big, __shfl_xor_sync(0xffffffffu, big, 2));
          big = max(big >> 16, big & 0xFFFFu);
          const bool finite = big < 0x7F80u;
          const int e = finite ? max(static_cast<int>(big >> 7) - 127, -100) : 0;
          constexpr int kExp = 21;
          const float up = __int_as_float((127 + kExp - e) << 23);
          int sum = 0;
#pragma unroll
          for (int j = 0; j < KW; ++j) {
            const uint32_t* p = reinterpret_cast<const uint32_t*>(&w[j]);
            // X + 128 (1 + 256 + 65536) has the digits plus 128 in its bytes; X comes out of an fp32 sum's low bits
            uint32_t y[8];
#pragma unroll
            for (int z = 0; z < 8; ++z) {  // dim 8 (KW t + j) + z
              const float v = __uint_as_float((z & 1) ? p[z >> 1] & 0xFFFF0000u : p[z >> 1] << 16);
              const uint32_t X = __float_as_uint(fmaf(v, up, 12582912.f)) - 0x4B400000u;  // (any, if not finite)
              sum += static_cast<int>(X);
              constexpr uint32_t kBias = 0x808080u;
              y[z] = (X + kBias) ^ kBias;
            }
            uint32_t b[3][2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {  // dims of the even codes, of the odd ones
              const uint32_t l0 = __byte_perm(y[z], y[z + 2], 0x5140), l1 = __byte_perm(y[z + 4], y[z + 6], 0x5140);
              const uint32_t h0 = __byte_perm(y[z], y[z + 2], 0x0062), h1 = __byte_perm(y[z + 4], y[z + 6], 0x0062);
              b[0][z] = __byte_perm(l0, l1, 0x5410);
              b[1][z] = __byte_perm(l0, l1, 0x7632);
              b[2][z] = __byte_perm(h0, h1, 0x5410);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              if constexpr (PACK) {
                b_at(n, j, 0, z) = g < 4 ? b[0][z] : b[1][z];
                b_at(n, j, 1, z) = b[2][z];
              } else {
#pragma unroll
                for (int y = 0; y < C::DT; ++y) b_at(n, j, y, z) = b[y][z];
              }
            }
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          // scores in base 2 from (16) sum X c
          const float down = __int_as_float((127 - (C::SPLIT ? 4 : 0) - kExp + e) << 23);
          const float sc = finite ? down * (A.scale * kLog2e) : NAN;
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int from = (col0 + z) * 4;
            qsum[n][z] = (C::SPLIT ? 16.f : 1.f) * static_cast<float>(__shfl_sync(0xffffffffu, sum, from));
            qsc[n][z] = __shfl_sync(0xffffffffu, sc, from);
            const int cc = c0 + 8 * n + col0 + z;
            const int p = cons.q.len - (cons.q.last - (cons.q.row0 + row_of(A, cc)));
            lim_hi[n][z] = cc < cols ? p + 1 : INT_MAX;
            lim_lo[n][z] = cc < cols ? window_begin(A, p) : 0;
            m[n][z] = -INFINITY;
            l[n][z] = zs[n][z] = 0.f;
          }
        }
        const int r_first = cons.q.row0 + row_of(A, c0);
        const int r_last = cons.q.row0 + row_of(A, min(c0 + C::COLS, cols) - 1);
        all_hi = cons.q.len - (cons.q.last - r_first) + 1;
        any_hi = cons.q.len - (cons.q.last - r_last) + 1;
        all_lo = window_begin(A, any_hi - 1);
        any_lo = window_begin(A, all_hi - 1);
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
      const unsigned char* stage = ring + slot * C::STAGEB;
      if (++slot == C::STAGES) slot = 0;
      // TILES tiles at a time; kept a loop, since a stage's whole code is more than the instruction cache likes.
#pragma unroll 1
      for (int sub = 0; sub < TOK / C::SUB; ++sub) {
        const unsigned char* st = stage + sub * TILES * C::TILEB;
        const uint32_t* kpar = reinterpret_cast<const uint32_t*>(stage + C::PAR) + sub * C::SUB;
        const uint32_t* vpar = kpar + TOK;
        const int tok0 = (cons.q.st0 + cons.tile) * TOK + sub * C::SUB;
        // a token of the step does not exist, or not every column sees every token
        bool odd = false;
#pragma unroll
        for (int z = 0; z < C::SUB; z += 32) odd |= (kpar[z + lane] & 0xFFFFu) == 0;
        odd = __any_sync(0xffffffffu, odd) || tok0 > all_hi - C::SUB || tok0 < all_lo;

        // scores in base 2: tokens tok_of[k] x columns col0, col0 + 1
        float s[TILES][NT][ROWS][2];
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          uint32_t wa[KW], wb[KW];
          const unsigned char *kt = st + j * C::TILEB + k_off, *kb = kt + 8 * C::ROWB;
          if constexpr (D == 64) {
            *reinterpret_cast<uint2*>(wa) = *reinterpret_cast<const uint2*>(kt);
            *reinterpret_cast<uint2*>(wb) = *reinterpret_cast<const uint2*>(kb);
          } else {
            *reinterpret_cast<uint4*>(wa) = *reinterpret_cast<const uint4*>(kt);
            *reinterpret_cast<uint4*>(wb) = *reinterpret_cast<const uint4*>(kb);
            if constexpr (D == 256) {
              *reinterpret_cast<uint4*>(wa + 4) = *reinterpret_cast<const uint4*>(kt + (k_off1 - k_off));
              *reinterpret_cast<uint4*>(wb + 4) = *reinterpret_cast<const uint4*>(kb + (k_off1 - k_off));
            }
          }
          int d[NT][C::DT][C::SPLIT ? 2 : 1][4] = {};  // sums over the even codes, the odd ones (16 times)
#pragma unroll
          for (int w = 0; w < KW; w += 2)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t a0, a1, a2, a3;
              if constexpr (C::SPLIT) {  // words w and w + 1, even or odd codes
                const uint32_t mask = e ? 0xF0F0F0F0u : 0x0F0F0F0Fu;
                a0 = wa[w] & mask, a1 = wb[w] & mask, a2 = wa[w + 1] & mask, a3 = wb[w + 1] & mask;
              } else {  // word w + e
                a0 = wa[w + e] & 0x0F0F0F0Fu, a1 = wb[w + e] & 0x0F0F0F0Fu;
                a2 = (wa[w + e] >> 4) & 0x0F0F0F0Fu, a3 = (wb[w + e] >> 4) & 0x0F0F0F0Fu;
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int y = 0; y < C::DT; ++y)
                  imma(d[n][y][C::SPLIT ? e : 0], a0, a1, a2, a3, qb[n][w / 2][y][e][0], qb[n][w / 2][y][e][1]);
            }
          // SPLIT: 16 sum d c, below 2^25 (256 dims: 2^26), so the three digits' sums are put together in fp32
          auto digit = [&](int n, int y, int z) {
            return C::SPLIT ? 16 * d[n][y][0][z] + d[n][y][C::SPLIT ? 1 : 0][z] : d[n][y][0][z];
          };
#pragma unroll
          for (int k = 0; k < ROWS; ++k) {
            const uint32_t par = kpar[16 * j + tok_of[k]];
            const float ks = sfd::half_bits_to_float(par & 0xFFFF), kz = sfd::half_bits_to_float(par >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                float f;  // sum X c, 16 times it if SPLIT
                if constexpr (PACK) {
                  // lanes t and t ^ 2 hold digits 0 and 1 of both tokens: each takes the other's of its own token
                  const int mine_a = digit(n, 0, z), mine_b = digit(n, 0, 2 + z);
                  const int other = __shfl_xor_sync(0xffffffffu, t < 2 ? mine_b : mine_a, 2);
                  f = fmaf(static_cast<float>(t < 2 ? mine_a : mine_b), own_w, static_cast<float>(other) * other_w);
                  f = fmaf(static_cast<float>(t < 2 ? digit(n, 1, z) : digit(n, 1, 2 + z)), 65536.f, f);
                } else {
                  f = C::SPLIT ? fmaf(static_cast<float>(digit(n, 1, 2 * k + z)), 256.f,
                                      static_cast<float>(digit(n, 0, 2 * k + z)))
                               : static_cast<float>(digit(n, 0, 2 * k + z) + 256 * digit(n, 1, 2 * k + z));
                  f = fmaf(static_cast<float>(digit(n, C::DT - 1, 2 * k + z)), 65536.f, f);
                }
                s[j][n][k][z] = fmaf(-kz, qsum[n][z], f) * (ks * qsc[n][z]);
              }
            if (odd) {
              const int tok = tok0 + 16 * j + tok_of[k];
              const bool there = (par & 0xFFFFu) != 0;
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int z = 0; z < 2; ++z)
                  if (!there || tok >= lim_hi[n][z] || tok < lim_lo[n][z]) s[j][n][k][z] = -INFINITY;
            }
          }
        }

        // the step's value scales and zero points
        float vs[TILES][ROWS], vz[TILES][ROWS], vmax = 0.f;
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
          for (int k = 0; k < ROWS; ++k) {
            uint32_t p = vpar[16 * j + tok_of[k]];
            if (odd) {  // a token that no column sees may hold anything
              const int tok = tok0 + 16 * j + tok_of[k];
              if (tok < any_lo || tok >= any_hi || (kpar[16 * j + tok_of[k]] & 0xFFFFu) == 0) p = 0;
            }
            vs[j][k] = sfd::half_bits_to_float(p & 0xFFFF);
            vz[j][k] = sfd::half_bits_to_float(p >> 16) - 8.f;
            vmax = fmaxf(vmax, fabsf(vs[j][k]));
          }

        // Raise the columns' references, and follow the largest value scale, when they have to: w = p v_s vscale stays
        // below 2^4 2^11.
        float top[NT][2];
        bool raise = vmax * vscale >= 2048.f || (vscale == 0.f && vmax > 0.f);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            top[n][z] = -INFINITY;
#pragma unroll
            for (int j = 0; j < TILES; ++j)
#pragma unroll
              for (int k = 0; k < ROWS; ++k) top[n][z] = fmaxf(top[n][z], s[j][n][k][z]);
            raise |= top[n][z] > m[n][z] + 4.f;
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, o));
          float grow = 1.f;
          if (vmax * vscale >= 2048.f || (vscale == 0.f && vmax > 0.f)) {
            // 2^(10 - exponent of vmax), exact
            const float next = __int_as_float((127 + 10 + 127 - (__float_as_int(vmax) >> 23)) << 23);
            if (vscale != 0.f) grow = next / vscale;
            vscale = next;
          }
          float alpha[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float mx = top[n][z];
#pragma unroll
              for (int o = PACK ? 2 : 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              mx = fmaxf(m[n][z], mx + 2.f);
              alpha[n][z] = mx == m[n][z] ? 1.f : ex2(m[n][z] - mx);  // 0 from -inf
              m[n][z] = mx;
              l[n][z] *= alpha[n][z];
              alpha[n][z] *= grow;
              zs[n][z] *= alpha[n][z];
            }
          if (!empty) {
            // the value product's columns 2t, 2t + 1 belong to the lane's score columns (packed: as weights or
            // remainders)
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                  acc[k][n][z] *= alpha[n][z & 1];
                }
            if (has_flushed) {
#pragma unroll 1
              for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float4& f = flushed[(k * NT + n) * 32];
                  const float4 x = f;
                  f = make_float4(x.x * alpha[n][0], x.y * alpha[n][1], x.z * alpha[n][0], x.w * alpha[n][1]);
                }
            }
          }
        }
        empty = false;

        // weights as operand fragments
        constexpr int WT = PACK ? 1 : 2;  // products of 8 columns per column tile
        uint32_t bw[TILES][NT][WT][2];
#pragma unroll
        for (int j = 0; j < TILES; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t hi2[ROWS], lo2[ROWS];
#pragma unroll
            for (int k = 0; k < ROWS; ++k) {
              float w[2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const float p = ex2(s[j][n][k][z] - (m[n][z] == -INFINITY ? 0.f : m[n][z]));
                l[n][z] += p;
                w[z] = p * (vs[j][k] * vscale);
                zs[n][z] = fmaf(w[z], vz[j][k], zs[n][z]);
              }
              const __half2 hh = __floats2half2_rn(w[0], w[1]);
              hi2[k] = reinterpret_cast<const uint32_t&>(hh);
              const float2 back = __half22float2(hh);
              lo2[k] = h2_bits(w[0] - back.x, w[1] - back.y);
            }
            if constexpr (PACK) {
              // columns 0-3 the weights, 4-7 the remainders: lanes t and t ^ 2 hold the two tokens of both
              const uint32_t y = __shfl_xor_sync(0xffffffffu, t < 2 ? lo2[0] : hi2[0], 2);
              bw[j][n][0][0] = transpose8x8(t < 2 ? hi2[0] : y);
              bw[j][n][0][1] = transpose8x8(t < 2 ? y : lo2[0]);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                bw[j][n][0][k] = transpose8x8(hi2[k]);
                bw[j][n][WT - 1][k] = transpose8x8(lo2[k]);
              }
            }
          }

        // values
#pragma unroll
        for (int j = 0; j < TILES; ++j) {
          uint32_t v[4][VW];  // tokens t, t + 4, t + 8, t + 12
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const unsigned char* vt = st + j * C::TILEB + ((z & 1) ? v_off1 : v_off0) + (z >> 1) * 8 * C::ROWB;
            if constexpr (D == 64)
              v[z][0] = *reinterpret_cast<const uint32_t*>(vt);
            else if constexpr (D == 128)
              *reinterpret_cast<uint2*>(v[z]) = *reinterpret_cast<const uint2*>(vt);
            else
              *reinterpret_cast<uint4*>(v[z]) = *reinterpret_cast<const uint4*>(vt);
          }
#pragma unroll
          for (int w = 0; w < VW; ++w)
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t x0 = __byte_perm(v[0][w], v[1][w], b | (4 + b) << 8);
              const uint32_t x1 = __byte_perm(v[2][w], v[3][w], b | (4 + b) << 8);
              const uint32_t a0 = nib_lo(x0), a1 = nib_hi(x0), a2 = nib_lo(x1), a3 = nib_hi(x1);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                hmma(acc[4 * w + b][n], a0, a1, a2, a3, bw[j][n][0][0], bw[j][n][0][1]);
                if constexpr (WT == 2)
                  hmma(acc[4 * w + b][n], a0, a1, a2, a3, bw[j][n][WT - 1][0], bw[j][n][WT - 1][1]);
              }
            }
        }
      }

      const bool ends = cons.tile + 1 == cons.q.stages || u + 1 == count;  // the segment's end, or the run's
      if (++since == C::FLUSH || (ends && has_flushed)) {
#pragma unroll
        for (int k = 0; k < MT; ++k)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float4& f = flushed[(k * NT + n) * 32];
            float(&x)[4] = acc[k][n];
            if (has_flushed) {
              const float4 y = f;
              x[0] += y.x, x[1] += y.y, x[2] += y.z, x[3] += y.w;
            }
            if (!ends) {
              f = make_float4(x[0], x[1], x[2], x[3]);
              x[0] = x[1] = x[2] = x[3] = 0.f;
            }
          }
        since = 0;
        has_flushed = true;
      }
      if (ends) {
        since = 0;
        has_flushed = false;
        const int seg_end = seg_at + cons.q.stages;
        const bool whole = seg_at >= 0 && seg_end <= count;
        const int which = seg_at < 0 ? 0 : 1;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int z = 0; z < 2; ++z) {
#pragma unroll
            for (int o = PACK ? 2 : 4; o < 32; o <<= 1) {
              l[n][z] += __shfl_xor_sync(0xffffffffu, l[n][z], o);
              zs[n][z] += __shfl_xor_sync(0xffffffffu, zs[n][z], o);
            }
            const float inv = l[n][z] == 0.f ? 0.f : 1.f / (l[n][z] * (vscale == 0.f ? 1.f : vscale));
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              if constexpr (PACK) {  // weights' and remainders' sums
                acc[k][n][z] += __shfl_xor_sync(0xffffffffu, acc[k][n][z], 2);
                acc[k][n][z + 2] += __shfl_xor_sync(0xffffffffu, acc[k][n][z + 2], 2);
              }
              acc[k][n][z] = (acc[k][n][z] - zs[n][z]) * inv;
              acc[k][n][z + 2] = (acc[k][n][z + 2] - zs[n][z]) * inv;
            }
          }
        }
        if (whole) {
          if (!PACK || t < 2) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int k = 0; k < MT; k += 2)
                  put<C>(A, cons.q.row0, cons.q.rows, cons.block, cons.h, 8 * n + col0 + z, D / 8 * g + 2 * k,
                         make_float4(acc[k][n][z], acc[k][n][z + 2], acc[k + 1][n][z], acc[k + 1][n][z + 2]));
          }
        } else {
          // At the run's end the drained ring has room for it; a part that comes before it goes to the workspace.
          __syncwarp();
          float* keep = u + 1 == count
                            ? reinterpret_cast<float*>(ring)
                            : W.heads + (static_cast<int64_t>(blockIdx.x) * C::WARPS + warp) * C::PART;
          if (!PACK || t < 2) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int col = 8 * n + col0 + z;
#pragma unroll
                for (int k = 0; k < MT; k += 2)
                  *reinterpret_cast<float4*>(keep + col * D + D / 8 * g + 2 * k) =
                      make_float4(acc[k][n][z], acc[k][n][z + 2], acc[k + 1][n][z], acc[k + 1][n][z + 2]);
                if (g == 0) keep[C::COLS * D + col] = l[n][z] == 0.f ? -INFINITY : m[n][z] + log2f(l[n][z]);
              }
          }
          if (lane == 0)
            parts[warp][which] =
                Part{lo + seg_at, lo + seg_end, keep, cons.q.row0, cons.q.rows, cons.block, cons.h};
        }
        fresh = true;
        seg_at = u + 1;
      }
      if (u + 1 < count) advance<C>(A, cons);
    }
  }

  // Segments that are split over the block's warps: the one begun in an earlier block, if any, then those begun in
  // each warp's run.  A warp per segment and column; lane k looks at part k.
  __syncthreads();
  static_assert(2 * C::WARPS <= 32, "a lane per part");
  const Part mine_p = lane < 2 * C::WARPS ? parts[lane >> 1][lane & 1] : Part{-1, 0, nullptr, 0, 0, 0, 0};
  const unsigned starts = __ballot_sync(0xffffffffu, mine_p.us >= b_lo && (lane & 1));
  const unsigned early_parts = __ballot_sync(0xffffffffu, mine_p.us >= 0 && mine_p.us < b_lo);
  if (warp == C::WARPS - 1) {
    const bool open = mine_p.us >= b_lo && mine_p.ue > b_hi && (lane & 1);
    if (open)
      W.tails[blockIdx.x] = Tail{1, mine_p.row0, mine_p.rows, mine_p.block, mine_p.h, runs.of(mine_p.ue - 1)};
    if (!__any_sync(0xffffffffu, open) && lane == 0) W.tails[blockIdx.x].open = 0;
  }
  const int chains = __popc(starts) + (early_parts != 0);
  for (int task = warp; task < chains * C::COLS; task += C::WARPS) {
    const int col = task % C::COLS;
    int nth = task / C::COLS;
    unsigned rest = starts;
    int from = __ffs(early_parts) - 1;
    if (early_parts == 0 || nth-- > 0) {
      for (int k = 0; k < nth; ++k) rest &= rest - 1;
      from = __ffs(rest) - 1;
    }
    const Part& p = parts[from >> 1][from & 1];
    const bool early = p.us < b_lo, late = p.ue > b_hi;
    const unsigned members = __ballot_sync(0xffffffffu, mine_p.us == p.us);
    // lane k: the k-th member
    const int n = __popc(members);
    rest = members;
    for (int k = 0; k < min(lane, n - 1); ++k) rest &= rest - 1;
    const int k_th = __ffs(rest) - 1;
    const float* at = parts[k_th >> 1][k_th & 1].at;
    const float lse = lane < n ? at[C::COLS * D + col] : -INFINITY;
    const float top = warp_top(lse);
    float sum = 0.f;
    float4 o[(D + 127) / 128] = {};
    join_column<C>(at, n, col, lse, top, sum, o);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    float* to = W.parts + (static_cast<int64_t>(blockIdx.x) * 2 + (early ? 0 : 1)) * C::PART;
#pragma unroll
    for (int z = 0; z < (D + 127) / 128; ++z) {
      const int dim = 4 * lane + 128 * z;
      if (dim >= D) continue;
      const float4 v = make_float4(o[z].x * inv, o[z].y * inv, o[z].z * inv, o[z].w * inv);
      if (!early && !late)
        put<C>(A, p.row0, p.rows, p.block, p.h, col, dim, v);
      else
        *reinterpret_cast<float4*>(to + col * D + dim) = v;
    }
    if ((early || late) && lane == 0) to[C::COLS * D + col] = sum == 0.f ? -INFINITY : top + log2f(sum);
  }
}

// Joins the parts of the segment that starts in block b and ends in a later one: JOIN warps per column, each taking
// every JOIN-th part, so that all their loads are on their way at once.
template <class C>
__global__ void __launch_bounds__(32 * C::COLS * C::JOIN) attn_paged_join_kernel(const __grid_constant__ Work W) {
  constexpr int D = C::D, Z = (D + 127) / 128;
  __shared__ float sum_sh[C::JOIN][C::COLS];
  __shared__ float4 o_sh[C::JOIN][C::COLS][Z][32];
  sfd::wait_for_previous();
  const Tail tail = W.tails[blockIdx.x];
  if (!tail.open) return;
  const int b = blockIdx.x, n = tail.last_cta - b + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = warp % C::COLS, share = warp / C::COLS;
  auto part = [&](int k) { return W.parts + (static_cast<int64_t>(b + k) * 2 + (k == 0 ? 1 : 0)) * C::PART; };
  float top = -INFINITY;
  for (int k = lane; k < n; k += 32) {
    const float v = part(k)[C::COLS * D + col];
    top = top != top || top > v ? top : v;
  }
  top = warp_top(top);
  float sum = 0.f;
  float4 o[Z] = {};
  const int mine = n > share ? (n - 1 - share) / C::JOIN + 1 : 0;  // parts share, share + JOIN, ...
  for (int k0 = 0; k0 < mine; k0 += 32) {
    const int k = share + C::JOIN * min(k0 + lane, mine - 1);
    const float lse = k0 + lane < mine ? part(k)[C::COLS * D + col] : -INFINITY;
    join_column<C>(part(k), min(32, mine - k0), col, lse, top, sum, o);
  }
#pragma unroll
  for (int z = 0; z < Z; ++z) o_sh[share][col][z][lane] = o[z];
  if (lane == 0) sum_sh[share][col] = sum;
  __syncthreads();
  if (share != 0) return;
#pragma unroll
  for (int v = 1; v < C::JOIN; ++v) {
    sum += sum_sh[v][col];
#pragma unroll
    for (int z = 0; z < Z; ++z) {
      const float4 x = o_sh[v][col][z][lane];
      o[z].x += x.x;
      o[z].y += x.y;
      o[z].z += x.z;
      o[z].w += x.w;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int z = 0; z < Z; ++z)
    if (4 * lane + 128 * z < D)
      put<C>(W.a, tail.row0, tail.rows, tail.block, tail.h, col, 4 * lane + 128 * z,
             make_float4(o[z].x * inv, o[z].y * inv, o[z].z * inv, o[z].w * inv));
}

// The workspace: tails, the blocks' parts, the warps' parts.
size_t tails_bytes(int blocks) { return (blocks * sizeof(Tail) + 255) / 256 * 256; }

template <class C>
struct Kernel {
  static size_t bytes(int blocks) {
    return tails_bytes(blocks) + static_cast<size_t>(blocks) * (2 + C::WARPS) * C::PART * sizeof(float);
  }
  static sf_status launch(const AttnArgs& A, void* ws, int blocks, cudaStream_t s) {
    Work W{};
    W.a = A;
    W.tails = static_cast<Tail*>(ws);
    W.parts = reinterpret_cast<float*>(static_cast<char*>(ws) + tails_bytes(blocks));
    W.heads = W.parts + static_cast<size_t>(blocks) * 2 * C::PART;
    W.blocks = blocks;
    static std::atomic<unsigned long long> told{0};
    sf_status st = sf::allow_smem(attn_paged_kernel<C>, C::SMEM, told);
    if (st != SF_OK) return st;
    st = sf::launch("attn_paged_kernel", attn_paged_kernel<C>, dim3(blocks), 32 * C::WARPS, C::SMEM, 1, s, W);
    if (st != SF_OK) return st;
    // its blocks start as the first kernel's end, and wait for the last
    return sf::launch("attn_paged_join_kernel", attn_paged_join_kernel<C>, dim3(blocks), 32 * C::COLS * C::JOIN, 0, 1,
                      s, W);
  }
};

// Calls f with the kernel for these sizes: 4 (packed), 8 or 16 columns a block, by the columns that a request's rows
// fill on average (rounded down: a padded batch has a few rows more than its requests; one padded to many more runs a
// wider kernel than it needs: right, but slower); d = 256 has no registers for 16.
template <class F>
auto with_kernel(int T, int R, int Hq, int Hkv, int d, F f) {
  const int64_t cols = static_cast<int64_t>(std::max(1, T / R)) * (Hq / Hkv);
  if (d == 64) {
    if (cols <= 4) return f(Kernel<Cfg<64, 1, true, 64, 12, 3>>{});
    if (cols <= 8) return f(Kernel<Cfg<64, 1, false, 64, 12, 3>>{});
    return f(Kernel<Cfg<64, 2, false, 64, 8, 3>>{});
  }
  if (d == 128) {
    if (cols <= 4) return f(Kernel<Cfg<128, 1, true, 64, 8, 2>>{});
    if (cols <= 8) return f(Kernel<Cfg<128, 1, false, 64, 8, 2>>{});
    return f(Kernel<Cfg<128, 2, false, 64, 8, 2>>{});
  }
  if (cols <= 4) return f(Kernel<Cfg<256, 1, true, 32, 8, 2>>{});
  return f(Kernel<Cfg<256, 1, false, 32, 8, 2>>{});
}

}  // namespace

extern "C" sf_status sf_attn_paged_workspace_size(int T, int R, int Hq, int Hkv, int d, size_t* bytes) {
  const char* what = "sf_attn_paged_workspace_size";
  SF_REQUIRE(bytes, "%s: null pointer", what);
  SF_REQUIRE(d == 64 || d == 128 || d == 256, "%s: d must be 64, 128 or 256", what);
  SF_REQUIRE(Hkv >= 1 && Hkv <= 256 && Hq >= Hkv && Hq % Hkv == 0 && Hq / Hkv <= 64,
             "%s: need Hkv in [1, 256] and Hq/Hkv a whole number up to 64", what);
  SF_REQUIRE(T >= 0 && R >= 1 && R <= 8192, "%s: need T >= 0 and R in [1, 8192]", what);
  const int blocks = sf::sm_count();
  auto size = [&](auto k) { return k.bytes(blocks); };
  *bytes = with_kernel(T, R, Hq, Hkv, d, size);
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
  SF_REQUIRE(static_cast<int64_t>(a->T) * (a->Hq / kv.Hkv) < (1 << 26), "%s: T * Hq/Hkv must be below 2^26", what);
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
  A.group = a->Hq / kv.Hkv;
  A.per_group = A.group == 1 ? 0 : static_cast<uint32_t>(((1ull << 32) + A.group - 1) / A.group);
  A.shift = sf::log2i(kv.page_size);
  A.num_pages = kv.num_pages;
  A.max_pages = a->max_pages;
  A.window = a->window;
  A.bf16_out = a->out_type == SF_BF16;
  auto run = [&](auto k) { return k.launch(A, a->workspace, sf::sm_count(), sf::as_cuda(stream)); };
  return with_kernel(a->T, a->R, a->Hq, kv.Hkv, kv.d, run);
}
