// Attention of a ragged batch over the 8-bit paged cache (bc_kv8_attention).
//
//   x_t = scale q.k_t, capped and biased as asked;  o = sum_t p_t v_t,
//   p = softmax(x) over the tokens the row sees,
// in one pass over the cache: running maximum m and sum l (base 2), o
// rescaled as the maximum grows.  Up to 64 query rows of a kv head share the
// bytes of its pages: up to 8 rows are 32 flops a byte, so HBM bounds them (64
// sequences of 1K to 8K tokens, 32 / 8 heads of 128, bf16: 454 MB in 78.6 us, 5.8
// TB/s, 7.1 while it streams); beyond, the work of a page and 8 rows does, one
// chain from its scores to its products on 3 warps a scheduler (16 sequences with
// 1 to 4 drafts of 4 rows, cap and window 4096: 111 MB in 44.6 us, half of the
// issue slots, 12% of the tensor pipe).  Times here are of graph replays; a call
// from Python takes 2 to 4 us more.
//
// Work split.  A segment is the pages of one (sequence, kv head, 8 query
// rows); the pages of all segments, in that order, are one line of units; it
// is cut into equal pieces, one per warp, whatever the lengths are: a warp's
// piece may begin and end inside a segment and hold several.  A CTA (one per
// SM) has 12 warps.  A warp reads its pages through a ring in shared memory,
// filled by bulk copies (a block of a page and head, scales included, is
// contiguous) 2 pages ahead, 24 blocks per SM (32 only lengthen the
// queues: 4 us more for 64 sequences of 1K to 8K tokens); the page numbers come
// from registers, 64 units ahead.  Sequences with more than 8 rows (several
// queries, or drafts) have their blocks read once per 8 rows, mostly from L2;
// the products, not the bytes, bound those (sharing a block between the warps
// of a sequence's rows left warps idle where sequences differ in queries: 11 us
// more for 16 sequences with 1 to 4 drafts in a window of 4096 tokens).
// A segment that lies in one warp's piece goes straight to the output.
// Pieces of a segment are merged in shared memory within a CTA, and through
// the scratch between CTAs, by the last of them to finish (an atomic ticket
// per segment, kept by the CTA it begins in; no spinning).  All merges run in
// a fixed order.
//
// Products on mma.sync m16n8k16 with f16 operands (both code types are exact
// in f16), the cache as the A operand and the 8 rows as its 8 columns, so no
// part of a tile is idle: S^T = K Q^T, then O^T = V^T P^T.  A tcgen05 tile
// would be 7/8 empty.  A row of q is scaled by a power of two so that its
// largest element is in [2^14, 2^15).  A bf16 q is exact in f16 (elements below
// 2^-31 of the largest: to 2^-39 of it), and weights of 11 bits serve a bf16
// output of 8 (a tenth of the outputs round to a neighbour of the nearest bf16
// number, with the error against 64 bits that 32-bit weights give, 1.7e-3 in the
// root mean square of the two cases above); for f32 both are split in two f16 numbers, hi + lo (22 bits, or
// as many as the smallest f16 number, 2^-24, leaves), for twice the products.
// The key scale multiplies the logit.  The value scale v of a page enters the
// weight, w = 2^(x + log2 v - mo + lift), with a second reference mo for x +
// log2 v: the f16 weight is then relative to the largest weight times scale
// seen, however far apart the scales are.  The references m and mo follow
// the maxima only when one is passed by more than 2^slack (one vote a page): the
// reductions over the lanes and the rescaling of o leave the usual path.  With
// slack 2 (f32) they do so a little more often than with 8: 0.2 us for four
// sequences of 16K to 128K tokens at half the pages (53.7 us).
//
// Fragment order.  Lane (g, t) = (lane / 4, lane % 4).  Dims are contracted
// in the order in which a lane finds them, 64u + 16t + 4w + 0..3 for step
// 4u + w (A and B alike).  Row n of score block j is token 4 (n / 2) + 2j +
// n % 2, so that after a transpose of 8 x 8 (movmatrix) lane (g, t) holds the
// weights of tokens 4t .. 4t + 3 for query row g: the B operand of the second
// product, whose A operand is one word (4 tokens of a dim) of the value
// codes, stored in that order.  Output block (v, i) holds dims 4 (8v + g) +
// 2i, + 2i + 1, so a lane ends with 4 neighbouring dims of rows 2t and 2t+1.
// Every shared-memory read is 16 bytes a lane, without bank conflicts.
#include "entry.h"
#include "kv8.cuh"

#include <math.h>
#include <algorithm>
#include <atomic>

namespace bc {

constexpr int kA8Warps = 12, kA8Threads = kA8Warps * 32;
constexpr int kA8Ring = 2;          // blocks in flight per warp
constexpr int kA8Rows = 8;          // query rows per segment
constexpr int kA8MaxCtas = 160;     // CTAs the scratch provides for
constexpr float kLog2e = 1.4426950408889634f;

struct Attn8Args {
  bc_kv8_attention_args a;
  float* part;            // [grid][2][8][HD + 4] partials between CTAs
  unsigned* tickets;      // [kA8MaxCtas] of the segment that begins in a CTA and goes on, zero between calls
  unsigned* status;       // bit 0: a wait gave up
};

// x / d for x < 2^31 and a quotient below 2^20: the float quotient is off by
// less than 1
__device__ __forceinline__ unsigned small_div(unsigned x, unsigned d) {
  unsigned q = (unsigned)__fdividef((float)x, (float)d);
  const int rest = (int)(x - q * d);
  if (rest < 0) --q;
  else if (rest >= (int)d) ++q;
  return q;
}

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {          // scales are 0, NaN or at least 2^-126
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// hi/lo f16 split of two floats
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_f16x2(x0, x1);
  const float2 h = __half22float2(*reinterpret_cast<__half2*>(&hi));
  lo = pack_f16x2(x0 - h.x, x1 - h.y);
}
__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A * B, 16 x 8 f32 accumulators, A two rows of words (a: row g, b: row
// g + 8; k order as B's)
__device__ __forceinline__ void mma_words(float* c, const uint32_t a[2], const uint32_t b[2], const uint32_t* q) {
  const uint32_t x[4] = {a[0], b[0], a[1], b[1]};
  mma_f16(c, x, q[0], q[1]);
}

// 8 x 8 f16 transpose over the warp
__device__ __forceinline__ uint32_t movm(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// cap * tanh(x / cap).  With bf16 outputs from the fast exponential and
// reciprocal, 1 - 2 / (1 + e^2t) with an error of 2^-23 or so, and for
// |t| < 0.1, where that would be relative to more than the result, from
// t - t^3 / 3 + 2 t^5 / 15 - 17 t^7 / 315 (next term below 10^-9 t).
template <bool PRECISE>
__device__ __forceinline__ float cap_logit(float x, float cap, float inv_cap) {
  if (PRECISE) return cap * tanhf(x / cap);
  const float t = x * inv_cap, u = t * t;
  float q;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(1.f + ex2(2.f * kLog2e * t)));
  const float p = x * fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return u < 0.01f ? p : fmaf(-2.f * cap, q, cap);
}

// the bytes of four e4m3 codes that are not numbers
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); }

// A segment as its flush and its masks need it.
struct Segment {
  int h, begin, r0;          // kv head, first unit, the sequence's first query row
  int row0, rows;            // its first row of the sequence's, and their end
  int first, last;           // positions of its first and last query
};

// References below every logit: nothing seen yet.
constexpr float kNoMax = -1e38f;
// A weight is at most 2^(slack + lift) = 2^15, within f16, and the largest at
// least 2^lift.  Half the smallest f16 number, 2^-25, is the error of a small one:
// 2^-32 of the largest under bf16 outputs, 2^-38 under f32 ones, whose references
// follow sooner for it.  The denominator sums weights of 32 bits, so that what
// lies below is lost from the output.
template <bool SPLIT>
struct Refs {
  static constexpr float slack = SPLIT ? 2.f : 8.f, lift = 15.f - slack;
};

// What a sequence needs of the cache.
struct Seq {
  int n;          // tokens
  int r0, own;    // first query row, its queries
  int lo, cnt;    // first page (without a list), pages (entries of the list)
  int rows;       // query rows of a kv head, max_q queries at most
};

__device__ __forceinline__ Seq seq_of(const bc_kv8_attention_args& a, int n, int r0, int own, int b) {
  Seq s;
  s.n = n;
  s.r0 = r0;
  s.own = max(own, 0);
  s.lo = s.cnt = 0;
  const int queries = min(s.own, a.max_q);
  s.rows = queries * a.group;
  if (queries == 0) return s;
  if (a.pages) {
    s.cnt = clampi(a.n_sel[b], 0, a.max_sel);
  } else {
    const int first = n - s.own, last = first + queries - 1;   // positions of the first and last query
    if (a.window > 0) s.lo = max(0, first - a.window + 1) / kPage;
    s.cnt = last < 0 ? 0 : max(0, last / kPage + 1 - s.lo);
  }
  return s;
}

// SPLIT: f32 queries and outputs (hi + lo operands); else bf16.  MODS: a cap
// or slopes.
template <int HD, int TYPE, bool SPLIT, bool MODS>
__global__ void __launch_bounds__(kA8Threads, 1) k_kv8_attn(const __grid_constant__ Attn8Args ga) {
  constexpr int BLK = kv8_block_bytes(HD);
  constexpr int U = HD / 64, V4 = HD / 32;
  constexpr int SROW = HD + 4;             // a partial's row: o, then m, l, mo
  constexpr float kSlack = Refs<SPLIT>::slack, kLift = Refs<SPLIT>::lift;
  const bc_kv8_attention_args& a = ga.a;
  const int B = a.batch, H = a.n_kv_heads, G = a.group;

  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;                                                     // [warps][kA8Ring] blocks
  float* heads = reinterpret_cast<float*>(smem + kA8Warps * kA8Ring * BLK); // [warps][kA8Rows][SROW]
  uint64_t* bars = reinterpret_cast<uint64_t*>(heads + kA8Warps * kA8Rows * SROW);
  int* s_cum = reinterpret_cast<int*>(bars + kA8Warps * kA8Ring);           // [B + 1] running sum of pages x tiles
  int* s_len = s_cum + B + 1;                                               // [B]
  int* s_row = s_len + B;                                                   // [B + 1] first query rows
  __shared__ int s_red[32];
  __shared__ int s_last[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const uint32_t full0 = smem_addr(bars) + 8 * warp * kA8Ring;
  if (tid < kA8Warps * kA8Ring) {
    mbar_init(smem_addr(bars) + 8 * tid, 1);
    mbar_init_fence();
  }
  pdl_wait();
  pdl_trigger();

  // ---- the line of units: every CTA sums the pages by itself
  const int ipt = (B + kA8Threads - 1) / kA8Threads;
  int mine = 0;
  for (int i = 0; i < ipt; ++i) {
    const int b = tid * ipt + i;
    if (b < B) {
      const int n = (int)min((long long)max(a.lens[b], 0), (long long)a.max_blocks * kPage);
      // bounds keep the differences inside an int whatever q_start holds
      const int r0 = a.q_start ? clampi(a.q_start[b], -(1 << 28), 1 << 29) : b;
      const int own = a.q_start ? clampi(a.q_start[b + 1], -(1 << 28), 1 << 29) - r0 : 1;
      s_len[b] = n;
      s_row[b] = r0;
      if (b == B - 1) s_row[B] = r0 + own;
      const Seq s = seq_of(a, n, r0, own, b);
      const int units = s.cnt * ((s.rows + kA8Rows - 1) / kA8Rows);
      s_cum[b] = units;
      mine += units;
    }
  }
  int T;
  int run = block_excl_scan<kA8Threads>(mine, s_red, &T);
  for (int i = 0; i < ipt; ++i) {
    const int b = tid * ipt + i;
    if (b < B) {
      const int units = s_cum[b];
      s_cum[b] = run;
      run += units;
    }
  }
  if (tid == 0) s_cum[B] = T;
  __syncthreads();

  // rows of sequences without pages
  for (int b = blockIdx.x; b < B; b += gridDim.x) {
    if (s_cum[b + 1] > s_cum[b]) continue;
    const int rows = min(max(s_row[b + 1] - s_row[b], 0), a.max_q);
    const int width = H * G * HD;
    for (int i = 0; i < rows; ++i) {
      const int row = s_row[b] + i;
      if (row < 0 || row >= a.n_q) continue;
      for (int e = tid; e < width; e += kA8Threads) {
        if (a.dtype == BC_F32) static_cast<float*>(a.out)[(size_t)row * width + e] = 0.f;
        else static_cast<__nv_bfloat16*>(a.out)[(size_t)row * width + e] = __float2bfloat16_rn(0.f);
      }
    }
  }

  const int total = T * H;
  const int per = max(1, (int)(((unsigned)total + gridDim.x * kA8Warps - 1) / (gridDim.x * kA8Warps)));   // units per warp
  const int per_cta = per * kA8Warps;
  const int c0 = (int)min((long long)blockIdx.x * per_cta, (long long)total);
  const int c1 = (int)min((long long)c0 + per_cta, (long long)total);
  if (c0 >= c1) return;
  const int g0 = (int)min((long long)c0 + (long long)warp * per, (long long)c1);
  const int g1 = (int)min((long long)g0 + per, (long long)c1);

  // row / G for the rows of a kv head (G <= 8, rows < 72): one multiplication
  const int g_inv = 65536 / G + 1;
  auto query_of = [&](int row) { return row * g_inv >> 16; };
  auto seq_at = [&](int b) { return seq_of(a, s_len[b], s_row[b], s_row[b + 1] - s_row[b], b); };
  // the segment of unit u: sequence, kv head, 8 rows, units
  auto locate = [&](int u, int& b, int& h, int& tile, int& begin, int& end) {
    int lo = 0, hi = B;                      // last b with s_cum[b] H <= u
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid] * H <= u) lo = mid;
      else hi = mid;
    }
    b = lo;
    const int tiles = (min(max(s_row[b + 1] - s_row[b], 0), a.max_q) * G + kA8Rows - 1) / kA8Rows;
    const unsigned of_head = s_cum[b + 1] - s_cum[b], at = u - s_cum[b] * H;
    const unsigned cnt = tiles == 1 ? of_head : of_head / (unsigned)tiles;
    h = small_div(at, of_head);
    tile = tiles == 1 ? 0 : small_div(at - h * of_head, cnt);
    begin = s_cum[b] * H + h * of_head + tile * cnt;
    end = begin + cnt;
  };

  // ---- pages of the cache: lane l holds those of units base + l and base +
  // 32 + l.  A lookup only starts its loads; found() turns what came into the
  // block number page * H + h and the page of the sequence, or -1 (not there).
  auto lookup = [&](int k, int& entry, int& logical) {
    entry = logical = -1;
    if (k >= g1 - g0) return;                    // (g0 + k might pass an int)
    const int u = g0 + k;
    int b, h, tile, begin, end;
    locate(u, b, h, tile, begin, end);
    if (a.pages) {
      logical = a.pages[((size_t)b * H + h) * a.max_sel + (u - begin)];
      if (logical < 0 || logical >= (s_len[b] + kPage - 1) / kPage) return;
    } else {
      logical = seq_at(b).lo + (u - begin);
    }
    entry = a.table[(size_t)b * a.max_blocks + logical];
  };
  auto found = [&](int k, int& block, int& logical) {
    int b, h, tile, begin, end;
    if (block >= 0 && block < a.n_pages) {
      locate(g0 + k, b, h, tile, begin, end);
      block = block * H + h;
    } else {
      block = logical = -1;
    }
  };
  int base = 0, bl0 = -1, bl1 = -1, lg0 = -1, lg1 = -1;

  const int n_units = g1 - g0;
  uint8_t* my_ring = ring + warp * kA8Ring * BLK;
  // the cache is read once: first to leave L2 (not so if it is read per 8 rows)
  uint64_t policy;
  if (G * a.max_q <= kA8Rows) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
  auto issue = [&](int k) {
    const int block = __shfl_sync(0xffffffffu, k - base < 32 ? bl0 : bl1, (k - base) & 31);
    if (lane == 0) {
      const uint32_t bar = full0 + 8 * (k & (kA8Ring - 1));
      if (block >= 0) {
        mbar_arrive_expect_tx(bar, BLK);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], "
            "%4;" ::"r"(smem_addr(my_ring + (k & (kA8Ring - 1)) * BLK)),
            "l"(static_cast<const uint8_t*>(a.pool) + (size_t)block * BLK), "r"(BLK), "r"(bar), "l"(policy)
            : "memory");
      } else {
        mbar_arrive(bar);                         // a page that is not there
      }
    }
  };

  // ---- the segment at hand
  // Lane (g, t) loads row g of its queries; scores, weights and outputs are of
  // rows 2t and 2t + 1.
  __shared__ Segment s_seg[kA8Warps];
  Segment* my_seg = s_seg + warp;
  int seg_end = g0;
  uint32_t qh[4 * U][2], ql[SPLIT ? 4 * U : 1][2];
  float o[V4][2][4];
  float m[2], l[2], mo[2], qs[2], slope[2];
  int at[2];                                  // the row's position (rows that are not there: INT32_MAX)
  int all_lo = 0, all_hi = 0;                 // positions every row sees
  int gave_up = -1;                           // a wait ran out: the pages issued until then

  constexpr int NRAW = SPLIT ? 4 * U : 2 * U;
  uint4 raw[NRAW];                        // query rows as loaded
  // takes up the segment of unit u and starts to load its queries
  auto begin_segment = [&](int u) {
    int b, h, tile, begin;
    locate(u, b, h, tile, begin, seg_end);
    const Seq s = seq_at(b);
    const int row0 = tile * kA8Rows, first = s.n - s.own;
    if (lane == 0) *my_seg = Segment{h, begin, s.r0, row0, s.rows, first, first + min(s.own, a.max_q) - 1};
    __syncwarp();
    #pragma unroll
    for (int v = 0; v < V4; ++v)
      #pragma unroll
      for (int i = 0; i < 4; ++i) o[v][0][i] = o[v][1][i] = 0.f;
    int w_lo = 0, w_hi = INT32_MAX;
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
      m[i] = mo[i] = kNoMax;
      l[i] = 0.f;
      const int row = row0 + 2 * t + i;
      at[i] = INT32_MAX;
      if (row < s.rows) {
        at[i] = first + query_of(row);
        if (a.window > 0) w_lo = max(w_lo, at[i] - a.window + 1);
        w_hi = min(w_hi, at[i]);
      }
      slope[i] = MODS && a.slopes && row < s.rows ? a.slopes[h * G + row - query_of(row) * G] : 0.f;
    }
    all_lo = __reduce_max_sync(0xffffffffu, w_lo);
    all_hi = __reduce_min_sync(0xffffffffu, w_hi);
    const int row = row0 + g, query = query_of(row), src = s.r0 + query;
    const bool ok = row < s.rows && src >= 0 && src < a.n_q;
    const size_t e0 = (size_t)(ok ? src : 0) * a.q_stride + (size_t)(ok ? (h - query) * G + row : 0) * HD + 16 * t;
    #pragma unroll
    for (int i = 0; i < NRAW; ++i) {
      const size_t e = e0 + (SPLIT ? 64 * (i / 4) + 4 * (i % 4) : 64 * (i / 2) + 8 * (i % 2));
      raw[i] = !ok ? make_uint4(0, 0, 0, 0)
                      : SPLIT ? *reinterpret_cast<const uint4*>(static_cast<const float*>(a.q) + e)
                              : *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + e);
    }
  };
  // turns the loaded queries into operands
  auto take_queries = [&]() {
    float x[16 * U];
    uint32_t top = 0;
    #pragma unroll
    for (int i = 0; i < NRAW; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (SPLIT) {
          x[4 * i + e] = __uint_as_float(w[e]);
        } else {
          x[8 * i + 2 * e] = bf16_lo(w[e]);
          x[8 * i + 2 * e + 1] = bf16_hi(w[e]);
        }
      }
    }
    #pragma unroll
    for (int d = 0; d < 16 * U; ++d) top = max(top, __float_as_uint(x[d]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = max((int)(top >> 23), 14);           // q 2^(141 - e) is below 2^15
    const float f = e == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(1.f, 141 - e);
    const float back = ldexpf(MODS ? a.scale : a.scale * kLog2e, e - 141);
    qs[0] = __shfl_sync(0xffffffffu, back, 8 * t);
    qs[1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
    #pragma unroll
    for (int w = 0; w < 4 * U; ++w)
      #pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float y0 = x[4 * w + 2 * i] * f, y1 = x[4 * w + 2 * i + 1] * f;
        if (SPLIT) split_f16(y0, y1, qh[w][i], ql[w][i]);
        else qh[w][i] = pack_f16x2(y0, y1);
      }
  };

  // Value codes that are not numbers, on a page that not every row sees: a row
  // that sees one becomes NaN in its dim, and the code 0, so that the rows that
  // mask it get 0 times a number.  (The append writes no such code.)
  auto take_out_nan = [&](uint8_t* blk, int pos0) {
    #pragma unroll
    for (int v = 0; v < V4; ++v) {
      uint4* x = reinterpret_cast<uint4*>(blk + kPage * HD + (8 * v + g) * 64 + t * 16);
      const uint4 y = *x;
      const uint32_t n0 = nan_codes(y.x), n1 = nan_codes(y.y), n2 = nan_codes(y.z), n3 = nan_codes(y.w);
      *x = make_uint4(y.x & ~n0, y.y & ~n1, y.z & ~n2, y.w & ~n3);
      #pragma unroll 1
      for (int r = 0; r < kA8Rows; ++r) {
        const int at0 = __shfl_sync(0xffffffffu, at[0], r >> 1), at1 = __shfl_sync(0xffffffffu, at[1], r >> 1);
        const int p = r & 1 ? at1 : at0;                  // the row's position
        uint32_t sees = 0;
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int token = pos0 + 4 * t + j;
          if (token <= p && (a.window == 0 || token > p - a.window)) sees |= 0xffu << (8 * j);
        }
        uint32_t hit = (n0 & sees ? 1u : 0u) | (n1 & sees ? 2u : 0u) | (n2 & sees ? 4u : 0u) | (n3 & sees ? 8u : 0u);
        hit |= __shfl_xor_sync(0xffffffffu, hit, 1);
        hit |= __shfl_xor_sync(0xffffffffu, hit, 2);
        #pragma unroll
        for (int d = 0; d < 4; ++d)
          #pragma unroll
          for (int i = 0; i < 2; ++i)
            if (r == 2 * t + i && (hit >> d & 1u)) o[v][d >> 1][2 * (d & 1) + i] = __uint_as_float(0x7fc00000u);
      }
    }
  };

  const float inv_cap = MODS && a.cap > 0.f ? 1.f / a.cap : 0.f;
  auto process = [&](uint8_t* blk, int lp) {
    const float* sc = reinterpret_cast<const float*>(blk + 2 * kPage * HD);
    const float ks = sc[0], lvs = lg2(sc[1]);
    float ca[4], cb[4];
    #pragma unroll
    for (int i = 0; i < 4; ++i) ca[i] = cb[i] = 0.f;
    {
      const uint8_t* kp = blk + (4 * (g >> 1) + (g & 1)) * 64 + t * 16;
      #pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint4 x = *reinterpret_cast<const uint4*>(kp + u * (kPage * 64));
        const uint4 y = *reinterpret_cast<const uint4*>(kp + u * (kPage * 64) + 128);
        const uint32_t xx[4] = {x.x, x.y, x.z, x.w}, yy[4] = {y.x, y.y, y.z, y.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[2], q[2];
          Kv8Code<TYPE>::decode(xx[i], p[0], p[1]);
          Kv8Code<TYPE>::decode(yy[i], q[0], q[1]);
          mma_words(SPLIT || !(i & 1) ? ca : cb, p, q, qh[4 * u + i]);
          if (SPLIT) mma_words(cb, p, q, ql[4 * u + i]);
        }
      }
    }
    // this lane's scores: rows 2t + i, tokens 4 (g / 2) + 2j + g % 2
    const int pos0 = lp * kPage, pos = pos0 + 4 * (g >> 1) + (g & 1);
    const bool whole = pos0 >= all_lo && pos0 + kPage - 1 <= all_hi;
    float c[2][2], y[2][2];
    bool passed = false;
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float f = qs[i] * ks;
      #pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = (ca[2 * j + i] + cb[2 * j + i]) * f;
        if (MODS) {
          if (a.cap > 0.f) x = cap_logit<SPLIT>(x, a.cap, inv_cap);
          if (a.slopes) x -= slope[i] * (float)(at[i] - (pos + 2 * j));   // a row that is not there: 0
          x *= kLog2e;
        }
        c[i][j] = x;
      }
    }
    if (!whole) {
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 2; ++j)
          if (pos + 2 * j > at[i] || (a.window > 0 && pos + 2 * j <= at[i] - a.window)) c[i][j] = -INFINITY;
    }
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
      y[i][0] = c[i][0] - m[i];
      y[i][1] = c[i][1] - m[i];
      passed |= fmaxf(y[i][0], y[i][1]) > fminf(kSlack, kSlack - lvs - (m[i] - mo[i]));
    }
    if (__any_sync(0xffffffffu, passed)) {
      float ao[2];
      #pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = fmaxf(c[i][0], c[i][1]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float m_new = fmaxf(m[i], mx), mo_new = fmaxf(mo[i], mx + lvs);
        l[i] *= ex2(m[i] - m_new);
        ao[i] = ex2(mo[i] - mo_new);
        m[i] = m_new;
        mo[i] = mo_new;
        y[i][0] = c[i][0] - m_new;
        y[i][1] = c[i][1] - m_new;
      }
      #pragma unroll
      for (int v = 0; v < V4; ++v)
        #pragma unroll
        for (int i = 0; i < 2; ++i) {
          o[v][i][0] *= ao[0];
          o[v][i][1] *= ao[1];
          o[v][i][2] *= ao[0];
          o[v][i][3] *= ao[1];
        }
    }
    // A scale that is not a number makes even a weight of 0 one.
    float w[2][2], z[2];
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
      z[i] = lvs + (m[i] - mo[i]) + kLift;
      const float f = ex2(z[i]);
      #pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p = ex2(y[i][j]);
        l[i] += p;
        w[i][j] = p * f;
      }
    }
    // A factor near or past the largest number, of values that make up for
    // logits far below the row's others: the weight from one exponent.  (Up to
    // 2^96 a p that is cut to 0 stands for less than f16 holds.)
    if (__any_sync(0xffffffffu, fmaxf(z[0], z[1]) > 96.f)) {
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 2; ++j) w[i][j] = ex2(y[i][j] + z[i]);
    }
    if (!whole) {
      // masked tokens weigh nothing, whatever the scales are (a key scale
      // that is not a number was replaced with the score)
      #pragma unroll
      for (int i = 0; i < 2; ++i)
        #pragma unroll
        for (int j = 0; j < 2; ++j)
          if (c[i][j] == -INFINITY) w[i][j] = 0.f;
      // value codes of tokens that no query sees may be any bytes: zero them
      // where this lane reads them
      const int any_lo = a.window > 0 ? my_seg->first - a.window + 1 : 0, any_hi = my_seg->last;
      uint32_t keep = 0xffffffffu;
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        if (pos0 + 4 * t + j < any_lo || pos0 + 4 * t + j > any_hi) keep &= ~(0xffu << (8 * j));
      bool odd = false;
      #pragma unroll 1
      for (int v = 0; v < V4; ++v) {
        uint4* x = reinterpret_cast<uint4*>(blk + kPage * HD + (8 * v + g) * 64 + t * 16);
        const uint4 y = make_uint4(x->x & keep, x->y & keep, x->z & keep, x->w & keep);
        if (TYPE == BC_KV8_E4M3) odd |= (nan_codes(y.x) | nan_codes(y.y) | nan_codes(y.z) | nan_codes(y.w)) != 0;
        *x = y;
      }
      if (TYPE == BC_KV8_E4M3 && __any_sync(0xffffffffu, odd)) take_out_nan(blk, pos0);
      // these stores come before the next copy into this block
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    uint32_t ph[2], pl[2];
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (SPLIT) {
        split_f16(w[0][j], w[1][j], ph[j], pl[j]);
        pl[j] = movm(pl[j]);
      } else {
        ph[j] = pack_f16x2(w[0][j], w[1][j]);
      }
      ph[j] = movm(ph[j]);
    }
    #pragma unroll
    for (int v = 0; v < V4; ++v) {
      const uint4 x = *reinterpret_cast<const uint4*>(blk + kPage * HD + (8 * v + g) * 64 + t * 16);
      const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
      #pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t p[2], q[2];
        Kv8Code<TYPE>::decode(ww[2 * i], p[0], p[1]);
        Kv8Code<TYPE>::decode(ww[2 * i + 1], q[0], q[1]);
        // The tensor cores cut sums off: a chain of them over the pages of a
        // piece is low by up to 2^-24 a page, nothing to bf16 outputs (a tenth of
        // a rounding at 8192 pages) but 1.8e-4 at 4096 pages to f32 ones, whose
        // pages are therefore added to nearest (6e-6; 82.7 against 79.7 us for 64
        // f32 sequences of 1K to 8K tokens, 53.4 against 52.9 for four of 16K to
        // 128K at half the pages).
        if (SPLIT) {
          float part[4] = {0.f, 0.f, 0.f, 0.f};
          mma_words(part, p, q, ph);
          mma_words(part, p, q, pl);
          #pragma unroll
          for (int e = 0; e < 4; ++e) o[v][i][e] += part[e];
        } else {
          mma_words(o[v][i], p, q, ph);
        }
      }
    }
  };

  // out = (o 2^-kLift / l) 2^(mo - m), two factors since one alone could fall
  // below the normal numbers; nothing seen: 0
  auto final_factor = [](float mm, float ll, float mmo) {
    return ll == 0.f ? make_float2(0.f, 0.f) : make_float2(exp2f(-kLift) / ll, exp2f(mmo - mm));
  };
  auto times = [](float4 y, float2 f) {
    return make_float4(y.x * f.x * f.y, y.y * f.x * f.y, y.z * f.x * f.y, y.w * f.x * f.y);
  };
  auto put = [&](int row, int j, int d, float4 y) {       // 4 dims of query row `row`, head j
    const size_t e = ((size_t)row * H * G + j) * HD + d;
    if (SPLIT) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + e) = y;
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + e) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    }
  };
  // the warp's rows: to a partial's rows at dst, or (dst null) to the output
  auto flush = [&](float* dst) {
    const Segment s = *my_seg;
    #pragma unroll
    for (int i = 0; i < 2; ++i) {
      float ll = l[i];
      ll += __shfl_xor_sync(0xffffffffu, ll, 4);
      ll += __shfl_xor_sync(0xffffffffu, ll, 8);
      ll += __shfl_xor_sync(0xffffffffu, ll, 16);
      if (gave_up >= 0) ll = __uint_as_float(0x7fc00000u);
      const int in = 2 * t + i, row = s.row0 + in;
      const float2 f = final_factor(m[i], ll, mo[i]);
      const int query = query_of(row), src = s.r0 + query;
      const bool ok = row < s.rows && src >= 0 && src < a.n_q;
      #pragma unroll
      for (int v = 0; v < V4; ++v) {
        const float4 y = make_float4(o[v][0][i], o[v][0][2 + i], o[v][1][i], o[v][1][2 + i]);
        const int d = 4 * (8 * v + g);
        if (dst) *reinterpret_cast<float4*>(dst + in * SROW + d) = y;
        else if (ok) put(src, (s.h - query) * G + row, d, times(y, f));
      }
      if (dst && g == 0) {
        float* ml = dst + in * SROW + HD;
        ml[0] = m[i];
        ml[1] = ll;
        ml[2] = mo[i];
      }
    }
    __syncwarp();
  };
  float* my_head = heads + warp * kA8Rows * SROW;

  // Segments cut between warps of this CTA, or between CTAs.  A cut segment's
  // pieces here: the tail of the warp it begins in (or the head of warp 0 if
  // it began in another CTA), then the heads of the next.  Lane w + 1 looks at
  // warp w's last segment, lane 0 at the CTA's first,
  // while the first pages are on their way.
  struct Cut {
    int b, h, s0, s1, first, last;   // segment, its units, the warps that hold pieces
    int cta0, cta1;                  // the CTAs it begins and ends in
    int row0, rows;                  // its first row, and how many
    bool from_tail;
  };
  __shared__ Cut s_cut[kA8Warps + 1];
  __shared__ int s_ncut, s_nout, s_out_cut[2];   // cuts; bit i: slot i's segment goes on in another CTA
  auto find_cuts = [&]() {
    if (warp == kA8Warps - 1) {
      const int w = lane - 1;
      const int e0 = (int)min((long long)c0 + (long long)max(w, 0) * per, (long long)c1);
      const int e1 = (int)min((long long)e0 + per, (long long)c1);
      Cut c;
      bool cut = w < kA8Warps && e0 < e1;
      if (cut) {
        int tile;
        locate(w < 0 ? c0 : e1 - 1, c.b, c.h, tile, c.s0, c.s1);
        cut = w < 0 ? c.s0 < c0 : c.s0 >= e0 && c.s1 > e1;
        c.first = max(w, 0);
        c.last = min(kA8Warps - 1, (int)small_div(min(c.s1, c1) - 1 - c0, per));
        c.cta0 = small_div(c.s0, per_cta);
        c.cta1 = small_div(c.s1 - 1, per_cta);
        c.row0 = tile * kA8Rows;
        c.rows = min(kA8Rows, min(max(s_row[c.b + 1] - s_row[c.b], 0), a.max_q) * G - c.row0);
        c.from_tail = w >= 0;
      }
      const unsigned mask = __ballot_sync(0xffffffffu, cut);
      const int at = __popc(mask & ((1u << lane) - 1));
      const bool head_out = cut && c.s0 < c0, tail_out = cut && !head_out && c.s1 > c1;
      if (cut) s_cut[at] = c;
      if (head_out) s_out_cut[0] = at;
      if (tail_out) s_out_cut[1] = at;
      const unsigned ho = __ballot_sync(0xffffffffu, head_out), to = __ballot_sync(0xffffffffu, tail_out);
      if (lane == 0) {
        s_ncut = __popc(mask);
        s_nout = (ho ? 1 : 0) | (to ? 2 : 0);
      }
    }
  };

  if (n_units > 0) begin_segment(g0);
  {
    lookup(lane, bl0, lg0);
    if (n_units > 32) lookup(32 + lane, bl1, lg1);
    found(lane, bl0, lg0);
    if (n_units > 32) found(32 + lane, bl1, lg1);
  }
  #pragma unroll 1
  for (int i = 0; i < min(kA8Ring, n_units); ++i) issue(i);
  if (n_units > 0) take_queries();
  find_cuts();
  #pragma unroll 1
  for (int k = 0;; ++k) {
    if (k == n_units || g0 + k == seg_end) {
      if (k == n_units && gave_up >= 0) {
        if (lane == 0) atomicOr(ga.status, 1u);
        // copies still in flight land before the ring is used again
        for (int i = max(0, gave_up - kA8Ring); i < gave_up; ++i)
          mbar_wait(full0 + 8 * (i & (kA8Ring - 1)), (i / kA8Ring) & 1);
      }
      if (k > 0) {
        const bool head = my_seg->begin < g0;
        float* dst = head ? my_head : nullptr;
        if (k == n_units && !head && seg_end > g1) {
          dst = reinterpret_cast<float*>(my_ring);       // the tail: the ring is idle now
        }
        flush(dst);
      }
      if (k == n_units) break;
      begin_segment(g0 + k);
      take_queries();
    }
    if ((k & 31) == 0 && k > 0) {
      base = k;
      bl0 = bl1;
      lg0 = lg1;
      lookup(k + 32 + lane, bl1, lg1);
    }
    if ((k & 31) == 16 && k > 16) found(k + 16 + lane, bl1, lg1);      // the loads are back
    const int lp = __shfl_sync(0xffffffffu, lg0, k & 31), stage = k & (kA8Ring - 1);
    if (gave_up < 0) {
      const bool ok = mbar_wait(full0 + 8 * stage, (k / kA8Ring) & 1);
      if (!__all_sync(0xffffffffu, ok)) gave_up = min(n_units, k + kA8Ring);
    }
    if (gave_up < 0 && lp >= 0) process(my_ring + stage * BLK, lp);
    __syncwarp();
    if (k + kA8Ring < n_units && gave_up < 0) issue(k + kA8Ring);
  }
  __syncthreads();

  // ---- merge the pieces of cut segments
  constexpr int D4 = HD / 4;
  const int tile_rows = min(kA8Rows, G * a.max_q), per_seg = tile_rows * D4;
  for (int e = tid; e < s_ncut * per_seg; e += kA8Threads) {
    const int which = small_div(e, per_seg), row = (e - which * per_seg) / D4, d = e % D4 * 4;
    const Cut& c = s_cut[which];
    if (row >= c.rows) continue;
    auto piece = [&](int x) {
      return (c.from_tail && x == c.first ? reinterpret_cast<const float*>(ring + x * kA8Ring * BLK)
                                          : heads + x * kA8Rows * SROW) + row * SROW;
    };
    float M = kNoMax, MO = kNoMax, L = 0.f;
    #pragma unroll 4
    for (int x = c.first; x <= c.last; ++x) {
      const float4 ml = *reinterpret_cast<const float4*>(piece(x) + HD);
      M = fmaxf(M, ml.x);
      MO = fmaxf(MO, ml.z);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    #pragma unroll 4
    for (int x = c.first; x <= c.last; ++x) {
      const float* q = piece(x);
      const float4 ml = *reinterpret_cast<const float4*>(q + HD);
      const float4 y = *reinterpret_cast<const float4*>(q + d);
      L += ex2(ml.x - M) * ml.y;
      const float f = ex2(ml.z - MO);
      acc.x += f * y.x; acc.y += f * y.y; acc.z += f * y.z; acc.w += f * y.w;
    }
    if (c.s0 >= c0 && c.s1 <= c1) {
      const int of_seq = c.row0 + row, query = query_of(of_seq), src = s_row[c.b] + query;
      const float2 f = final_factor(M, L, MO);
      if (src >= 0 && src < a.n_q)
        put(src, (c.h - query) * G + of_seq, d, times(acc, f));
    } else {
      float* dst = ga.part + ((blockIdx.x * 2 + (c.s0 < c0 ? 0 : 1)) * kA8Rows + row) * SROW;
      *reinterpret_cast<float4*>(dst + d) = acc;
      if (d == 0) *reinterpret_cast<float4*>(dst + HD) = make_float4(M, L, MO, 0.f);
    }
  }
  if (!s_nout) return;

  // ---- the last CTA of a cut segment merges its partials
  __syncthreads();
  if (tid < 2) {
    bool last = false;
    if (s_nout >> tid & 1) {
      const Cut& c = s_cut[s_out_cut[tid]];
      unsigned* ticket = ga.tickets + c.cta0;
      unsigned prev;
      asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(prev) : "l"(ticket) : "memory");
      last = prev == (unsigned)(c.cta1 - c.cta0);
      if (last) *ticket = 0u;
    }
    s_last[tid] = last;
  }
  __syncthreads();
  if (!s_last[0] && !s_last[1]) return;
  float* s_fac = reinterpret_cast<float*>(ring);        // [2][kA8Rows][partials]
  float2* s_out = reinterpret_cast<float2*>(s_fac + 2 * kA8Rows * kA8MaxCtas);      // [2][kA8Rows]
  // partial of row `row` in the x-th CTA of segment c, which begins in the first one
  auto partial = [&](const Cut& c, int x, int row) {
    return ga.part + (((c.cta0 + x) * 2 + (x == 0 ? 1 : 0)) * kA8Rows + row) * SROW;
  };
  // both slots at once: a warp a row for the weights, then a thread 4 dims
  for (int ir = warp; ir < 2 * kA8Rows; ir += kA8Warps) {
    const int i = ir / kA8Rows, row = ir % kA8Rows;
    if (!s_last[i]) continue;
    const Cut& c = s_cut[s_out_cut[i]];
    if (row >= c.rows) continue;
    const int n_c = c.cta1 - c.cta0 + 1;
    float M = kNoMax, MO = kNoMax, L = 0.f;
    float4 ml[kA8MaxCtas / 32];
    #pragma unroll
    for (int j = 0; j < kA8MaxCtas / 32; ++j) {
      ml[j] = make_float4(kNoMax, 0.f, kNoMax, 0.f);
      if (32 * j + lane < n_c) ml[j] = __ldcg(reinterpret_cast<const float4*>(partial(c, 32 * j + lane, row) + HD));
      M = fmaxf(M, ml[j].x);
      MO = fmaxf(MO, ml[j].z);
    }
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, o));
    }
    #pragma unroll
    for (int j = 0; j < kA8MaxCtas / 32; ++j) {
      L += ex2(ml[j].x - M) * ml[j].y;
      if (32 * j + lane < n_c) s_fac[ir * kA8MaxCtas + 32 * j + lane] = ex2(ml[j].z - MO);
    }
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_out[ir] = final_factor(M, L, MO);
  }
  __syncthreads();
  for (int e = tid; e < 2 * per_seg; e += kA8Threads) {
    const int i = e >= per_seg, row = (e - i * per_seg) / D4, d = e % D4 * 4;
    if (!s_last[i]) continue;
    const Cut& c = s_cut[s_out_cut[i]];
    if (row >= c.rows) continue;
    const int n_c = c.cta1 - c.cta0 + 1, ir = i * kA8Rows + row;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < n_c; x0 += 8) {               // 8 partials in flight, the last ones too
      float4 y[8];
      #pragma unroll
      for (int j = 0; j < 8; ++j)
        y[j] = x0 + j < n_c ? __ldcg(reinterpret_cast<const float4*>(partial(c, x0 + j, row) + d))
                            : make_float4(0.f, 0.f, 0.f, 0.f);
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (x0 + j >= n_c) break;
        const float f = s_fac[ir * kA8MaxCtas + x0 + j];
        acc.x += f * y[j].x; acc.y += f * y[j].y; acc.z += f * y[j].z; acc.w += f * y[j].w;
      }
    }
    const int of_seq = c.row0 + row, query = query_of(of_seq), src = s_row[c.b] + query;
    const float2 f = s_out[ir];
    if (src >= 0 && src < a.n_q)
      put(src, (c.h - query) * G + of_seq, d, times(acc, f));
  }
}

}  // namespace bc

using namespace bc;

static bool attn8_sizes_ok(int batch, int H, int group, int max_q, int hd) {
  return batch >= 1 && batch <= BC_RAGGED_MAX_BATCH && H >= 1 && H <= 65535 && group >= 1 && group <= 8 && max_q >= 1 &&
         max_q <= 64 && group * max_q <= 64 && (hd == 64 || hd == 128);
}

// Scratch: the status word, the tickets, the partials between CTAs.  The words
// that have to be zero lie in the same place whatever the sizes are, so calls
// of different sizes can share a scratch.
constexpr size_t kA8TicketsAt = 256, kA8PartAt = 1024;
static_assert(kA8TicketsAt + 4 * kA8MaxCtas <= kA8PartAt, "tickets overlap the partials");

template <int HD, int TYPE, bool SPLIT, bool MODS>
static cudaError_t attn8_launch(const Attn8Args& g, int grid, cudaStream_t st) {
  auto kern = k_kv8_attn<HD, TYPE, SPLIT, MODS>;
  const size_t fixed = kA8Warps * (kA8Ring * (kv8_block_bytes(HD) + 8ull) + 4ull * kA8Rows * (HD + 4));
  // once per device: the most that any batch needs
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(fixed + 4ull * (3 * BC_RAGGED_MAX_BATCH + 2)));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev);
  }
  return launch_op(kern, dim3(grid), dim3(kA8Threads), fixed + 4ull * (3 * (size_t)g.a.batch + 2), st, g);
}

extern "C" size_t bc_kv8_attention_scratch_bytes(int batch, int n_kv_heads, int group, int max_q, int head_dim) {
  if (!attn8_sizes_ok(batch, n_kv_heads, group, max_q, head_dim)) return 0;
  return kA8PartAt + 4ull * kA8MaxCtas * 2 * kA8Rows * (head_dim + 4);
}

extern "C" bc_status bc_kv8_attention(const bc_kv8_attention_args* a, void* stream) {
  const char* who = "bc_kv8_attention";
  if (!a) return entry_fail(BC_EINVAL, "%s: null arguments", who);
  if (!a->q || !a->out || !a->pool || !a->lens || !a->table || !a->scratch || !a->pages != !a->n_sel)
    return entry_fail(BC_EINVAL, "%s: null pointer", who);
  if (a->head_dim != 64 && a->head_dim != 128) return entry_fail(BC_EINVAL, "%s: head_dim must be 64 or 128", who);
  if (!attn8_sizes_ok(a->batch, a->n_kv_heads, a->group, a->max_q, a->head_dim))
    return entry_fail(BC_EINVAL, "%s: need batch in [1, %d], group in [1, 8] and 1 <= group * max_q <= 64", who,
                      BC_RAGGED_MAX_BATCH);
  if (a->dtype != BC_F32 && a->dtype != BC_BF16) return entry_fail(BC_EINVAL, "%s: bad dtype %d", who, (int)a->dtype);
  if (a->type != BC_KV8_E4M3 && a->type != BC_KV8_INT8)
    return entry_fail(BC_EINVAL, "%s: bad code type %d", who, (int)a->type);
  if (a->n_pages < 1 || a->n_pages > INT32_MAX / kPage || a->max_blocks < 1 || a->max_blocks > 1 << 25 ||
      a->n_q < 0 || a->n_q > 1 << 29 || (a->pages && a->max_sel < 1))
    return entry_fail(BC_EINVAL, "%s: bad page or row counts", who);
  if ((long long)a->n_pages * a->n_kv_heads > INT32_MAX)
    return entry_fail(BC_EINVAL, "%s: more than 2^31 - 1 blocks in the pool", who);
  const int tiles = (a->group * a->max_q + kA8Rows - 1) / kA8Rows;
  if ((long long)a->batch * a->n_kv_heads * std::max(a->max_blocks, a->pages ? a->max_sel : 0) > INT32_MAX / tiles)
    return entry_fail(BC_EINVAL, "%s: too many pages over all sequences, heads and rows", who);
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->pool, 16))
    return entry_fail(BC_EINVAL, "%s: q, out and pool must be 16-byte aligned", who);
  if (a->q_stride % 8 || a->q_stride < (long long)a->n_kv_heads * a->group * a->head_dim)
    return entry_fail(BC_EINVAL, "%s: q_stride must be a multiple of 8 and cover the heads", who);
  if (!aligned(a->scratch, 256)) return entry_fail(BC_EINVAL, "%s: scratch must be 256-byte aligned", who);
  // a cap below the normal range has no finite reciprocal
  if (!(a->cap == 0.f || (a->cap >= 1.17549435e-38f && a->cap <= 3.4e38f)) || a->window < 0 ||
      !(fabsf(a->scale) <= 3.4e38f))
    return entry_fail(BC_EINVAL, "%s: cap must be 0 or a positive normal number, window not negative, scale finite", who);
  if (a->scratch_bytes < bc_kv8_attention_scratch_bytes(a->batch, a->n_kv_heads, a->group, a->max_q, a->head_dim))
    return entry_fail(BC_ENOMEM, "%s: scratch too small", who);
  if (a->n_q == 0) return BC_OK;
  const bool f32 = a->dtype == BC_F32;
  Attn8Args g;
  g.a = *a;
  // a window that reaches every token is none
  if (a->window >= (long long)a->max_blocks * kPage + 64) g.a.window = 0;
  char* sc = static_cast<char*>(a->scratch);
  g.status = reinterpret_cast<unsigned*>(sc);
  g.tickets = reinterpret_cast<unsigned*>(sc + kA8TicketsAt);
  g.part = reinterpret_cast<float*>(sc + kA8PartAt);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return entry_cuda(e, who);
  const int grid = std::max(1, std::min(sms, kA8MaxCtas));
  const bool mods = a->cap > 0.f || a->slopes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define A8M(HD, TY, R) (mods ? attn8_launch<HD, TY, R, true>(g, grid, st) : attn8_launch<HD, TY, R, false>(g, grid, st))
#define A8R(HD, TY) (f32 ? A8M(HD, TY, true) : A8M(HD, TY, false))
#define A8T(HD) (a->type == BC_KV8_E4M3 ? A8R(HD, 0) : A8R(HD, 1))
  e = a->head_dim == 128 ? A8T(128) : A8T(64);
#undef A8T
#undef A8R
#undef A8M
  return entry_cuda(e, who);
}

extern "C" bc_status bc_kv8_attention_status(void* scratch, void* stream) {
  const char* who = "bc_kv8_attention_status";
  if (!scratch) return entry_fail(BC_EINVAL, "%s: null scratch", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, scratch, sizeof word, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return entry_cuda(e, who);
  if (!word) return BC_OK;
  e = cudaMemsetAsync(scratch, 0, sizeof word, st);
  if (e != cudaSuccess) return entry_cuda(e, who);
  return entry_fail(BC_ETIMEOUT, "%s: a wait for a copy gave up", who);
}
