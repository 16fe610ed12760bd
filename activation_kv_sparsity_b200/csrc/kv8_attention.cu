// Attention of a ragged batch over the 8-bit paged cache (bc_kv8_attention).
//
//   x_t = scale q.k_t, capped and biased as asked;  o = sum_t p_t v_t,
//   p = softmax(x) over the tokens the row sees,
// in one pass over the cache: running maximum m and sum l (base 2), o
// rescaled as the maximum grows.  Up to 64 query rows of a kv head share the
// bytes of its pages: 1 byte per key or value element read once, at most 128
// flops for it, so HBM bounds it.
//
// Work split.  The pages of all (sequence, kv head) pairs, in that order, are
// one line of units; it is cut into equal pieces, one per worker, whatever
// the lengths are: a worker's piece may begin and end inside a sequence and
// hold several.  A CTA (one per SM) has 8 warps; NT warps that take 8 or 16
// query rows each form a worker and share its pages.  A worker reads its
// pages through a ring in shared memory, filled by bulk copies (a block of a
// page and head, scales included, is contiguous) 4 NT pages ahead, 32 blocks
// per SM; the page numbers come from registers, 64 units ahead.
// A segment that lies in one worker's piece goes straight to the output.
// Pieces of a segment are merged in shared memory within a CTA, and through
// the scratch between CTAs, by the last of them to finish (an atomic ticket
// per pair, no spinning).  All merges run in a fixed order.
//
// Products on mma.sync m16n8k16 with f16 operands: both code types are exact
// in f16.  8 or 16 rows would leave 7/8 of a tcgen05 tile empty.  A row of q
// is scaled by a power of two so that its largest element is in [1/2, 1) and
// split in two f16 numbers, q = hi + lo (22 bits; a bf16 q is exact in hi
// down to 2^-24 of its largest element); the weights likewise.  With up to 8
// rows the two parts are the upper and the lower half of one A operand; 16
// rows (bf16 only) take the first part alone, 11 bits against the 8 of the
// output.
// The key scale multiplies the logit.  The value scale v of a page enters the
// weight's exponent, w = 2^(x + log2 v - mo + 8), with a second running
// maximum mo of x + log2 v: the f16 weight is then relative to the largest
// weight times scale seen, however far apart the scales are, and 8 more bits
// lie above f16's subnormals.
//
// Fragment order.  Lane (g, t) = (lane / 4, lane % 4).  Keys: dims are
// contracted in the order in which a lane finds them, 64u + 16t + 4w + 0..3
// for step 4u + w (A and B alike).  The score columns are tokens in such an
// order, 4 (n / 2) + 2j + n % 2 for column n of block j, that lane t holds
// tokens 4t .. 4t + 3 of row g; that is the A operand of the second product
// whose B operand is one word (4 tokens of a dim) of the value codes, which
// are stored in that order, and the output block 4v + j holds dims
// 4 (8v + n) + j.  Every shared-memory read is 16 bytes a lane, 512
// contiguous ones a warp.
#include "entry.h"
#include "kv8.cuh"

#include <algorithm>
#include <atomic>

namespace bc {

constexpr int kA8Warps = 8;
constexpr int kA8Threads = kA8Warps * 32;
constexpr int kA8Stages = 32;       // blocks in flight per CTA
constexpr int kA8MaxCtas = 160;     // CTAs the scratch provides for
constexpr float kLog2e = 1.4426950408889634f;

struct Attn8Args {
  bc_kv8_attention_args a;
  int nt;                 // warps per worker
  int rows;               // group * max_q
  float* part;            // [grid][2][rows][HD + 4] partials between CTAs
  unsigned* tickets;      // [batch * n_kv_heads], zero between calls
  unsigned* status;       // bit 0: a wait gave up
};

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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

// 2^x relative to a maximum that may still be -inf (nothing seen)
__device__ __forceinline__ float finite_or_0(float m) { return m == -INFINITY ? 0.f : m; }

// What a sequence needs of the cache.
struct Seq {
  int n;          // tokens
  int r0, own;    // first query row, its queries
  int lo, cnt;    // first page (without a list), pages (entries of the list)
};

__device__ __forceinline__ Seq seq_of(const bc_kv8_attention_args& a, int n, int r0, int own, int b) {
  Seq s;
  s.n = n;
  s.r0 = r0;
  s.own = max(own, 0);
  s.lo = s.cnt = 0;
  const int rows = min(s.own, a.max_q);
  if (rows == 0) return s;
  if (a.pages) {
    s.cnt = clampi(a.n_sel[b], 0, a.max_sel);
  } else {
    const int first = n - s.own, last = first + rows - 1;   // positions of the first and last query
    if (a.window > 0) s.lo = max(0, first - a.window + 1) / kPage;
    s.cnt = last < 0 ? 0 : max(0, last / kPage + 1 - s.lo);
  }
  return s;
}

template <int HD, int TYPE, bool R16, bool MODS>
__global__ void __launch_bounds__(kA8Threads, 1) k_kv8_attn(const __grid_constant__ Attn8Args ga) {
  constexpr int BLK = kv8_block_bytes(HD);
  constexpr int ROWS = R16 ? 16 : 8;       // query rows per warp
  constexpr int NR = R16 ? 2 : 1;          // rows per lane
  constexpr int U = HD / 64, V4 = HD / 32;
  constexpr int SROW = HD + 4;             // a partial's row: o, then m, l, mo
  const bc_kv8_attention_args& a = ga.a;
  const int B = a.batch, H = a.n_kv_heads, G = a.group, NT = ga.nt;
  const int GP = kA8Warps / NT, S = kA8Stages / GP;     // workers per CTA, ring stages per worker

  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  float* heads = reinterpret_cast<float*>(smem + kA8Stages * BLK);          // [GP][NT * ROWS][SROW]
  float* tails = reinterpret_cast<float*>(ring);                            // the same, once the ring is idle
  uint64_t* bars = reinterpret_cast<uint64_t*>(heads + kA8Warps * ROWS * SROW);   // full[32], empty[32]
  int* s_cum = reinterpret_cast<int*>(bars + 2 * kA8Stages);                // [B + 1] running sum of the pages
  int* s_len = s_cum + B + 1;                                               // [B]
  int* s_row = s_len + B;                                                   // [B + 1] first query rows
  __shared__ int s_red[32];
  __shared__ int s_last[2];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int worker = warp / NT, wt = warp % NT;
  const uint32_t full0 = smem_addr(bars) + 8 * worker * S, empty0 = full0 + 8 * kA8Stages;
  if (tid < kA8Stages) {
    mbar_init(smem_addr(bars) + 8 * tid, 1);
    mbar_init(smem_addr(bars) + 8 * (kA8Stages + tid), NT);
  }
  if (tid == 0) mbar_init_fence();
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
      const int r0 = a.q_start ? clampi(a.q_start[b], -(1 << 29), 1 << 30) : b;
      const int own = a.q_start ? clampi(a.q_start[b + 1], -(1 << 29), 1 << 30) - r0 : 1;
      s_len[b] = n;
      s_row[b] = r0;
      if (b == B - 1) s_row[B] = r0 + own;
      const int cnt = seq_of(a, n, r0, own, b).cnt;
      s_cum[b] = cnt;
      mine += cnt;
    }
  }
  int T;
  int run = block_excl_scan<kA8Threads>(mine, s_red, &T);
  for (int i = 0; i < ipt; ++i) {
    const int b = tid * ipt + i;
    if (b < B) {
      const int cnt = s_cum[b];
      s_cum[b] = run;
      run += cnt;
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
  const int per = max(1, (int)(((long long)total + gridDim.x * GP - 1) / (gridDim.x * GP)));   // units per worker
  const int per_cta = per * GP;
  const int c0 = (int)min((long long)blockIdx.x * per_cta, (long long)total);
  const int c1 = (int)min((long long)c0 + per_cta, (long long)total);
  if (c0 >= c1) return;
  const int g0 = (int)min((long long)c0 + (long long)worker * per, (long long)c1);
  const int g1 = (int)min((long long)g0 + per, (long long)c1);

  // the pair (b, h) that unit u belongs to, and the units of that pair
  auto locate = [&](int u, int& b, int& h, int& begin, int& end) {
    const int x = u / H;
    int lo = 0, hi = B;                      // last b with s_cum[b] <= x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid] <= x) lo = mid;
      else hi = mid;
    }
    b = lo;
    const int cnt = s_cum[b + 1] - s_cum[b], base = s_cum[b] * H;
    h = (u - base) / cnt;
    begin = base + h * cnt;
    end = begin + cnt;
  };
  auto seq_at = [&](int b) { return seq_of(a, s_len[b], s_row[b], s_row[b + 1] - s_row[b], b); };

  // ---- page numbers: lane l holds those of units base + l and base + 32 + l
  auto lookup = [&](int k, int& phys, int& logical) {
    phys = logical = -1;
    const int u = g0 + k;
    if (u >= g1) return;
    int b, h, begin, end;
    locate(u, b, h, begin, end);
    const int nblk = (s_len[b] + kPage - 1) / kPage;
    int lp;
    if (a.pages) {
      lp = a.pages[((size_t)b * H + h) * a.max_sel + (u - begin)];
      if (lp < 0 || lp >= nblk) return;
    } else {
      lp = seq_at(b).lo + (u - begin);
    }
    const int p = a.table[(size_t)b * a.max_blocks + lp];
    if (p < 0 || p >= a.n_pages) return;
    logical = lp;
    phys = p;
  };
  int base = 0, ph0, ph1, lg0, lg1;
  lookup(lane, ph0, lg0);
  lookup(32 + lane, ph1, lg1);
  auto phys_of = [&](int k) { return __shfl_sync(0xffffffffu, k - base < 32 ? ph0 : ph1, (k - base) & 31); };

  const int n_units = g1 - g0;
  const uint8_t* pool = static_cast<const uint8_t*>(a.pool);
  uint8_t* my_ring = ring + (size_t)worker * S * BLK;
  int is_b, is_h = 0, is_begin, is_end = g0;      // the pair of the unit issued last
  auto issue = [&](int k) {                       // by the leader warp, all lanes
    const int p = phys_of(k);
    const int u = g0 + k;
    if (u >= is_end) locate(u, is_b, is_h, is_begin, is_end);
    if (lane == 0) {
      const uint32_t bar = full0 + 8 * (k & (S - 1));
      if (p >= 0) {
        mbar_arrive_expect_tx(bar, BLK);
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                smem_addr(my_ring + (size_t)(k & (S - 1)) * BLK)),
            "l"(pool + ((size_t)p * H + is_h) * BLK), "r"(BLK), "r"(bar)
            : "memory");
      } else {
        mbar_arrive(bar);                         // a page that is not there
      }
    }
  };
  int issued = 0;
  if (wt == 0)
    for (; issued < min(S, n_units); ++issued) issue(issued);

  // ---- the segment at hand
  int b = 0, h = 0, seg_begin = g0, seg_end = g0;
  int r0 = 0, seg_rows = 0;
  uint32_t qa[4 * U][4];
  float o[4 * V4][4];
  float m[NR], l[NR], mo[NR], qs[NR], slope[NR];
  int lo[NR], hi[NR];                         // positions the row sees
  int tile_lo = 0, tile_hi = 0;               // positions every row of the warp sees
  int any_lo = 0, any_hi = 0;                 // positions some row of the warp sees
  bool live = false, dead = false;

  auto begin_segment = [&](int u) {
    locate(u, b, h, seg_begin, seg_end);
    const Seq s = seq_at(b);
    r0 = s.r0;
    seg_rows = min(s.own, a.max_q) * G;
    live = wt * ROWS < seg_rows;
    #pragma unroll
    for (int i = 0; i < 4 * V4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    #pragma unroll
    for (int r = 0; r < NR; ++r) {
      m[r] = mo[r] = -INFINITY;
      l[r] = 0.f;
    }
    if (!live) return;
    int w_lo = 0, w_hi = INT32_MAX, s_lo = INT32_MAX, s_hi = -1;
    #pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = wt * ROWS + g + 8 * r, i = row / G, j = h * G + row % G;
      const int src = r0 + i;
      const bool ok = row < seg_rows && src >= 0 && src < a.n_q;
      const int p = s.n - s.own + i;
      lo[r] = 0;
      hi[r] = INT32_MAX;
      if (row < seg_rows) {
        hi[r] = p;
        lo[r] = a.window > 0 ? max(0, p - a.window + 1) : 0;
        w_lo = max(w_lo, lo[r]);
        w_hi = min(w_hi, hi[r]);
        s_lo = min(s_lo, lo[r]);
        s_hi = max(s_hi, hi[r]);
      }
      slope[r] = MODS && a.slopes && row < seg_rows ? a.slopes[j] : 0.f;
      float x[U][16];
      uint32_t top = 0;
      #pragma unroll
      for (int c = 0; c < U; ++c) {
        #pragma unroll
        for (int d = 0; d < 16; ++d) x[c][d] = 0.f;
        if (ok) {
          const size_t at = (size_t)src * a.q_stride + (size_t)j * HD + 64 * c + 16 * t;
          if (a.dtype == BC_F32) {
            #pragma unroll
            for (int d = 0; d < 16; d += 4) {
              const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at + d);
              x[c][d] = y.x; x[c][d + 1] = y.y; x[c][d + 2] = y.z; x[c][d + 3] = y.w;
            }
          } else {
            #pragma unroll
            for (int d = 0; d < 16; d += 8) {
              const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) + at + d);
              const uint32_t w[4] = {y.x, y.y, y.z, y.w};
              #pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[c][d + 2 * e] = bf16_lo(w[e]);
                x[c][d + 2 * e + 1] = bf16_hi(w[e]);
              }
            }
          }
        }
        #pragma unroll
        for (int d = 0; d < 16; ++d) top = max(top, __float_as_uint(x[c][d]) & 0x7fffffffu);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int e = (int)(top >> 23);                    // q 2^(126 - e) is below 1
      const float f = e == 255 ? __uint_as_float(0x7fc00000u) : ldexpf(1.f, 126 - e);
      qs[r] = ldexpf(MODS ? a.scale : a.scale * kLog2e, e - 126);
      #pragma unroll
      for (int c = 0; c < U; ++c)
        #pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float* y = x[c] + 4 * w;
          if (R16) {
            qa[4 * c + w][r] = pack_f16x2(y[0] * f, y[1] * f);
            qa[4 * c + w][2 + r] = pack_f16x2(y[2] * f, y[3] * f);
          } else {
            split_f16(y[0] * f, y[1] * f, qa[4 * c + w][0], qa[4 * c + w][1]);
            split_f16(y[2] * f, y[3] * f, qa[4 * c + w][2], qa[4 * c + w][3]);
          }
        }
    }
    tile_lo = __reduce_max_sync(0xffffffffu, w_lo);
    tile_hi = __reduce_min_sync(0xffffffffu, w_hi);
    any_lo = __reduce_min_sync(0xffffffffu, s_lo);
    any_hi = __reduce_max_sync(0xffffffffu, s_hi);
  };

  auto process = [&](const uint8_t* blk, int lp) {
    const float* sc = reinterpret_cast<const float*>(blk + 2 * kPage * HD);
    const float ks = sc[0], lvs = log2f(sc[1]);
    float c[2][4];
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
      const uint8_t* kp = blk + (4 * (g >> 1) + 2 * j + (g & 1)) * 64 + t * 16;
      #pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint4 w = *reinterpret_cast<const uint4*>(kp + u * (kPage * 64));
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          Kv8Code<TYPE>::decode(ww[i], b0, b1);
          mma_f16(c[j], qa[4 * u + i], b0, b1);
        }
      }
    }
    const int pos0 = lp * kPage;
    const bool whole = pos0 >= tile_lo && pos0 + kPage - 1 <= tile_hi;
    float w[NR][4];
    bool rescale = false;
    float ao[NR];
    #pragma unroll
    for (int r = 0; r < NR; ++r) {
      float x[4];
      if (R16) {
        x[0] = c[0][2 * r]; x[1] = c[0][2 * r + 1]; x[2] = c[1][2 * r]; x[3] = c[1][2 * r + 1];
      } else {
        x[0] = c[0][0] + c[0][2]; x[1] = c[0][1] + c[0][3]; x[2] = c[1][0] + c[1][2]; x[3] = c[1][1] + c[1][3];
      }
      const float f = qs[r] * ks;
      bool see[4];
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] *= f;
        const int pos = pos0 + 4 * t + j;
        if (MODS) {
          if (a.cap > 0.f) x[j] = a.cap * tanhf(x[j] / a.cap);
          // a row that is not there has hi = INT32_MAX and no slope
          if (a.slopes) x[j] -= slope[r] * (float)(hi[r] - pos);
          x[j] *= kLog2e;
        }
        see[j] = whole || (pos >= lo[r] && pos <= hi[r]);
        if (!see[j]) x[j] = -INFINITY;
      }
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[r], mx), m_use = finite_or_0(m_new);
      const float mo_new = fmaxf(mo[r], mx + lvs), mo_use = finite_or_0(mo_new);
      const float al = ex2(m[r] - m_use);
      ao[r] = ex2(mo[r] - mo_use);
      rescale |= mo_new > mo[r];
      m[r] = m_new;
      mo[r] = mo_new;
      const float shift = lvs - mo_use + 8.f;
      float sum = 0.f;
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        float p = ex2(x[j] - m_use);
        w[r][j] = ex2(x[j] + shift);
        if (!see[j]) p = w[r][j] = 0.f;          // whatever the scales are
        sum += p;
      }
      l[r] = l[r] * al + sum;
    }
    if (__any_sync(0xffffffffu, rescale)) {
      #pragma unroll
      for (int i = 0; i < 4 * V4; ++i) {
        o[i][0] *= ao[0];
        o[i][1] *= ao[0];
        o[i][2] *= ao[NR - 1];
        o[i][3] *= ao[NR - 1];
      }
    }
    uint32_t pa[4];
    if (R16) {
      pa[0] = pack_f16x2(w[0][0], w[0][1]);
      pa[1] = pack_f16x2(w[NR - 1][0], w[NR - 1][1]);
      pa[2] = pack_f16x2(w[0][2], w[0][3]);
      pa[3] = pack_f16x2(w[NR - 1][2], w[NR - 1][3]);
    } else {
      split_f16(w[0][0], w[0][1], pa[0], pa[1]);
      split_f16(w[0][2], w[0][3], pa[2], pa[3]);
    }
    // value codes of tokens that no row sees may be any bytes: zero them
    uint32_t keep = 0xffffffffu;
    if (!whole) {
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int pos = pos0 + 4 * t + j;
        if (pos < any_lo || pos > any_hi) keep &= ~(0xffu << (8 * j));
      }
    }
    #pragma unroll
    for (int v = 0; v < V4; ++v) {
      const uint4 x = *reinterpret_cast<const uint4*>(blk + kPage * HD + (8 * v + g) * 64 + t * 16);
      const uint32_t ww[4] = {x.x & keep, x.y & keep, x.z & keep, x.w & keep};
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b0, b1;
        Kv8Code<TYPE>::decode(ww[j], b0, b1);
        mma_f16(o[4 * v + j], pa, b0, b1);
      }
    }
  };

  // out = o / l 2^(mo - m - 8); nothing seen: 0
  auto final_factor = [](float mm, float ll, float mmo) {
    if (ll == 0.f) return 0.f;
    return mmo == -INFINITY && ll == ll ? 0.f : exp2f(finite_or_0(mmo) - finite_or_0(mm) - 8.f) / ll;
  };
  auto put = [&](int row, int j, int d, float4 y) {       // 4 dims of query row `row`, head j
    const size_t at = ((size_t)row * H * G + j) * HD + d;
    if (a.dtype == BC_F32) {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
    } else {
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
          make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    }
  };
  // the warp's rows: to a partial's rows at dst, or (dst null) to the output
  auto flush = [&](float* dst) {
    if (!live) return;
    #pragma unroll
    for (int r = 0; r < NR; ++r) {
      float ll = l[r];
      ll += __shfl_xor_sync(0xffffffffu, ll, 1);
      ll += __shfl_xor_sync(0xffffffffu, ll, 2);
      if (dead) ll = __uint_as_float(0x7fc00000u);
      const int row = wt * ROWS + g + 8 * r;
      const float f = final_factor(m[r], ll, mo[r]);
      const int i = row / G, src = r0 + i;
      const bool ok = row < seg_rows && src >= 0 && src < a.n_q;
      #pragma unroll
      for (int v = 0; v < V4; ++v)
        #pragma unroll
        for (int half = 0; half < 2; ++half) {
          float y[4];
          #pragma unroll
          for (int j = 0; j < 4; ++j)
            y[j] = R16 ? o[4 * v + j][2 * r + half] : o[4 * v + j][half] + o[4 * v + j][2 + half];
          const int d = 32 * v + 8 * t + 4 * half;
          if (dst)
            *reinterpret_cast<float4*>(dst + (size_t)row * SROW + d) = make_float4(y[0], y[1], y[2], y[3]);
          else if (ok)
            put(src, h * G + row % G, d, make_float4(y[0] * f, y[1] * f, y[2] * f, y[3] * f));
        }
      if (dst && t == 0) {
        float* ml = dst + (size_t)row * SROW + HD;
        ml[0] = m[r];
        ml[1] = ll;
        ml[2] = mo[r];
      }
    }
  };
  float* my_head = heads + (size_t)worker * NT * ROWS * SROW;

  const int lag = NT == 1 ? 0 : 1;
  bool tail = false;
  for (int k = 0; k < n_units; ++k) {
    if (g0 + k == seg_end) {
      if (k > 0) flush(seg_begin < g0 ? my_head : nullptr);
      begin_segment(g0 + k);
    }
    if (k == base + 32) {
      base += 32;
      ph0 = ph1;
      lg0 = lg1;
      lookup(base + 32 + lane, ph1, lg1);
    }
    const int lp = __shfl_sync(0xffffffffu, lg0, k - base);
    const int stage = k & (S - 1);
    if (!dead && !mbar_wait(full0 + 8 * stage, (k / S) & 1)) dead = true;
    dead = __any_sync(0xffffffffu, dead);
    if (live && !dead && lp >= 0) process(my_ring + (size_t)stage * BLK, lp);
    __syncwarp();
    if (NT > 1 && lane == 0) mbar_arrive(empty0 + 8 * stage);
    const int old = k - lag;                            // its stage is free again
    if (wt == 0 && old >= 0 && old + S < n_units) {
      if (NT > 1 && !dead && !mbar_wait(empty0 + 8 * (old & (S - 1)), (old / S) & 1)) dead = true;
      dead = __any_sync(0xffffffffu, dead);
      if (!dead) {
        issue(old + S);
        issued = old + S + 1;
      }
    }
  }
  if (n_units > 0) {
    if (seg_begin < g0) flush(my_head);
    else if (seg_end <= g1) flush(nullptr);
    else tail = true;
  }
  if (dead) {
    // copies still in flight land before the ring is used again
    if (lane == 0) atomicOr(ga.status, 1u);
    if (wt == 0)
      for (int k = max(0, issued - S); k < issued; ++k) mbar_wait(full0 + 8 * (k & (S - 1)), (k / S) & 1);
  }
  __syncthreads();
  if (tail) flush(tails + (size_t)worker * NT * ROWS * SROW);
  __syncthreads();

  // ---- segments cut between workers of this CTA, or between CTAs
  // A cut segment's pieces here: the tail of the worker it begins in (or the
  // head of worker 0 if it began in another CTA), then the heads of the next.
  int n_cut = 0, cut_b[2], cut_h[2], cut_first[2], cut_count[2];
  for (int w = -1; w < GP; ++w) {
    int sb, sh, s0, s1;
    const int e0 = (int)min((long long)c0 + (long long)max(w, 0) * per, (long long)c1);
    const int e1 = (int)min((long long)e0 + per, (long long)c1);
    if (e0 >= e1) continue;
    locate(w < 0 ? c0 : e1 - 1, sb, sh, s0, s1);
    if (w < 0 ? s0 >= c0 : s0 < e0 || s1 <= e1) continue;
    const int w_first = max(w, 0), w_last = min(GP - 1, (min(s1, c1) - 1 - c0) / per);
    const bool here = s0 >= c0 && s1 <= c1;
    const int rows = min(max(s_row[sb + 1] - s_row[sb], 0), a.max_q) * G;
    const int slot = s0 < c0 ? 0 : 1;
    float* part = ga.part + ((size_t)blockIdx.x * 2 + slot) * ga.rows * SROW;
    for (int e = tid; e < rows * (HD / 4); e += kA8Threads) {
      const int row = e / (HD / 4), d = e % (HD / 4) * 4;
      auto piece = [&](int x) {
        return (w >= 0 && x == w ? tails : heads) + ((size_t)x * NT * ROWS + row) * SROW;
      };
      float M = -INFINITY, MO = -INFINITY, L = 0.f;
      for (int x = w_first; x <= w_last; ++x) {
        M = fmaxf(M, piece(x)[HD]);
        MO = fmaxf(MO, piece(x)[HD + 2]);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = w_first; x <= w_last; ++x) {
        const float* q = piece(x);
        L += ex2(q[HD] - finite_or_0(M)) * q[HD + 1];
        const float f = ex2(q[HD + 2] - finite_or_0(MO));
        const float4 y = *reinterpret_cast<const float4*>(q + d);
        acc.x += f * y.x; acc.y += f * y.y; acc.z += f * y.z; acc.w += f * y.w;
      }
      if (here) {
        const int src = s_row[sb] + row / G;
        const float f = final_factor(M, L, MO);
        if (src >= 0 && src < a.n_q) put(src, sh * G + row % G, d, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
      } else {
        float* dst = part + (size_t)row * SROW;
        *reinterpret_cast<float4*>(dst + d) = acc;
        if (d == 0) *reinterpret_cast<float4*>(dst + HD) = make_float4(M, L, MO, 0.f);
      }
    }
    if (!here) {
      cut_b[slot] = sb;
      cut_h[slot] = sh;
      cut_first[slot] = s0 / per_cta;
      cut_count[slot] = (s1 - 1) / per_cta - s0 / per_cta + 1;
      n_cut |= 1 << slot;
    }
  }
  if (!n_cut) return;

  // ---- the last CTA of a cut segment merges its partials
  __syncthreads();
  if (tid < 2) {
    s_last[tid] = 0;
    if (n_cut >> tid & 1) {
      unsigned* ticket = ga.tickets + (size_t)cut_b[tid] * H + cut_h[tid];
      unsigned prev;
      asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(prev) : "l"(ticket) : "memory");
      s_last[tid] = prev == (unsigned)(cut_count[tid] - 1);
      if (s_last[tid]) *ticket = 0u;
    }
  }
  __syncthreads();
  #pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!s_last[i]) continue;
    const int sb = cut_b[i], n_c = cut_count[i];
    const int rows = min(max(s_row[sb + 1] - s_row[sb], 0), a.max_q) * G;
    // partial of the x-th CTA: the segment begins in the first one
    auto piece = [&](int x, int row) {
      return ga.part + (((size_t)cut_first[i] + x) * 2 + (x == 0 ? 1 : 0)) * ga.rows * SROW + (size_t)row * SROW;
    };
    for (int e = tid; e < rows * (HD / 4); e += kA8Threads) {
      const int row = e / (HD / 4), d = e % (HD / 4) * 4;
      float M = -INFINITY, MO = -INFINITY, L = 0.f;
      for (int x = 0; x < n_c; ++x) {
        const float4 ml = __ldcg(reinterpret_cast<const float4*>(piece(x, row) + HD));
        M = fmaxf(M, ml.x);
        MO = fmaxf(MO, ml.z);
      }
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = 0; x < n_c; ++x) {
        const float* q = piece(x, row);
        const float4 ml = __ldcg(reinterpret_cast<const float4*>(q + HD));
        const float4 y = __ldcg(reinterpret_cast<const float4*>(q + d));
        L += ex2(ml.x - finite_or_0(M)) * ml.y;
        const float f = ex2(ml.z - finite_or_0(MO));
        acc.x += f * y.x; acc.y += f * y.y; acc.z += f * y.z; acc.w += f * y.w;
      }
      const int src = s_row[sb] + row / G;
      const float f = final_factor(M, L, MO);
      if (src >= 0 && src < a.n_q)
        put(src, cut_h[i] * G + row % G, d, make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f));
    }
  }
}

}  // namespace bc

using namespace bc;

static bool attn8_sizes_ok(int batch, int H, int group, int max_q, int hd) {
  return batch >= 1 && batch <= BC_RAGGED_MAX_BATCH && H >= 1 && H <= 65535 && group >= 1 && group <= 8 && max_q >= 1 &&
         max_q <= 64 && group * max_q <= 64 && (hd == 64 || hd == 128);
}

// Scratch: the status word, the tickets, the partials between CTAs.
struct Attn8Layout {
  size_t tickets, part, total;
};
static Attn8Layout attn8_layout(int batch, int H, int rows, int hd) {
  Attn8Layout y;
  y.tickets = 256;
  y.part = y.tickets + ((4ull * batch * H + 255) & ~255ull);
  y.total = y.part + 4ull * kA8MaxCtas * 2 * rows * (hd + 4);
  return y;
}

template <int HD, int TYPE, bool R16, bool MODS>
static cudaError_t attn8_launch(const Attn8Args& g, int grid, cudaStream_t st) {
  auto kern = k_kv8_attn<HD, TYPE, R16, MODS>;
  const size_t fixed = (size_t)kA8Stages * kv8_block_bytes(HD) + 4ull * kA8Warps * (R16 ? 16 : 8) * (HD + 4) +
                       16ull * kA8Stages;
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
  return attn8_layout(batch, n_kv_heads, group * max_q, head_dim).total;
}

extern "C" bc_status bc_kv8_attention(const bc_kv8_attention_args* a, void* stream) {
  const char* who = "bc_kv8_attention";
  if (!a) return entry_fail(BC_EINVAL, "%s: null arguments", who);
  if (!a->q || !a->out || !a->pool || !a->lens || !a->table || !a->scratch || (a->pages && !a->n_sel))
    return entry_fail(BC_EINVAL, "%s: null pointer", who);
  if (a->head_dim != 64 && a->head_dim != 128) return entry_fail(BC_EINVAL, "%s: head_dim must be 64 or 128", who);
  if (!attn8_sizes_ok(a->batch, a->n_kv_heads, a->group, a->max_q, a->head_dim))
    return entry_fail(BC_EINVAL, "%s: need batch in [1, %d], group in [1, 8] and 1 <= group * max_q <= 64", who,
                      BC_RAGGED_MAX_BATCH);
  if (a->dtype != BC_F32 && a->dtype != BC_BF16) return entry_fail(BC_EINVAL, "%s: bad dtype %d", who, (int)a->dtype);
  if (a->type != BC_KV8_E4M3 && a->type != BC_KV8_INT8)
    return entry_fail(BC_EINVAL, "%s: bad code type %d", who, (int)a->type);
  if (a->n_pages < 1 || a->n_pages > INT32_MAX / kPage || a->max_blocks < 1 || a->max_blocks > 1 << 26 ||
      a->n_q < 0 || a->n_q > 1 << 30 || (a->pages && a->max_sel < 1))
    return entry_fail(BC_EINVAL, "%s: bad page or row counts", who);
  if ((long long)a->batch * a->n_kv_heads * std::max(a->max_blocks, a->pages ? a->max_sel : 0) > INT32_MAX)
    return entry_fail(BC_EINVAL, "%s: more than 2^31 - 1 pages over all sequences and heads", who);
  if (!aligned(a->q, 16) || !aligned(a->out, 16) || !aligned(a->pool, 16))
    return entry_fail(BC_EINVAL, "%s: q, out and pool must be 16-byte aligned", who);
  if (a->q_stride % 8 || a->q_stride < (long long)a->n_kv_heads * a->group * a->head_dim)
    return entry_fail(BC_EINVAL, "%s: q_stride must be a multiple of 8 and cover the heads", who);
  if (!aligned(a->scratch, 256)) return entry_fail(BC_EINVAL, "%s: scratch must be 256-byte aligned", who);
  if (!(a->cap >= 0.f) || a->window < 0 || !(a->scale == a->scale))
    return entry_fail(BC_EINVAL, "%s: cap and window must not be negative, scale a number", who);
  if (a->scratch_bytes < bc_kv8_attention_scratch_bytes(a->batch, a->n_kv_heads, a->group, a->max_q, a->head_dim))
    return entry_fail(BC_ENOMEM, "%s: scratch too small", who);
  if (a->n_q == 0) return BC_OK;
  const bool f32 = a->dtype == BC_F32;
  Attn8Args g;
  g.a = *a;
  // a window that reaches every token is none
  if (a->window >= (long long)a->max_blocks * kPage + 64) g.a.window = 0;
  g.rows = a->group * a->max_q;
  // 8 rows a warp with both f16 parts of queries and weights; 16 rows with
  // the first part alone where the output is bf16 and 8 rows are not enough
  const bool r16 = !f32 && g.rows > 8;
  g.nt = 1;
  while (g.nt * (r16 ? 16 : 8) < g.rows) g.nt *= 2;
  const Attn8Layout y = attn8_layout(a->batch, a->n_kv_heads, g.rows, a->head_dim);
  char* sc = static_cast<char*>(a->scratch);
  g.status = reinterpret_cast<unsigned*>(sc);
  g.tickets = reinterpret_cast<unsigned*>(sc + y.tickets);
  g.part = reinterpret_cast<float*>(sc + y.part);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return entry_cuda(e, who);
  const int grid = std::max(1, std::min(sms, kA8MaxCtas));
  const bool mods = a->cap > 0.f || a->slopes;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
#define A8M(HD, TY, R) (mods ? attn8_launch<HD, TY, R, true>(g, grid, st) : attn8_launch<HD, TY, R, false>(g, grid, st))
#define A8R(HD, TY) (r16 ? A8M(HD, TY, true) : A8M(HD, TY, false))
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
