// Penalties, biases and grammar masks on logits (bc_logits_adjust): one pass
// over the logits, HBM-bound.
//
// Persistent CTAs take pieces of at most 8192 ids, neighbours of a row one
// after the other, and load a piece's logits (16 bytes a thread and round, as
// they are: a conversion on the way would wait for them) while the one before
// is worked on.  A row's history and biases are read once per row and CTA into
// shared memory.  For each piece the CTA walks them and marks the ids that fall
// into the piece, a word per id and list; each thread then looks its own ids up
// and clears their words.  A word of the history is bit 31, "seen in the
// prompt", and the count of the output tokens; a word of the biases the place of
// the last entry for the id (a maximum), so no result depends on the order of
// the atomics.
// Graph replays: 160 rows of 128256 f32 logits with histories of up to 8192
// tokens, 32 biases and masks take 41 us (4.0 TB/s of logits), 34 us with
// histories of up to 1000 tokens, 27 us with neither lists nor masks (6.0 TB/s,
// the copy's rate); in bf16 36, 28 and 12 us.  What the lists cost is the walks
// and the barriers around them: every piece of a row walks all of its lists.  Slower were a CTA a piece that walks the lists in L2 (68 us) and a
// copy and a scatter from hash tables (55); pieces in shared memory by
// asynchronous copies leave the lists too little room, and cutting a row's list to
// the CTA's own ids takes longer than the walks that it shortens.
#include "common.cuh"
#include "entry.h"

#include <algorithm>
#include <atomic>

namespace bc {

constexpr int kLogitThreads = 512;
constexpr int kLogitCtas = 2;                    // per SM
constexpr int kLogitWalk = 8;                    // further ones per thread in flight

// A piece: at most kRounds times 16 bytes a thread, held in registers.  Its two
// arrays of marks and the lists fill half an SM's shared memory.
template <typename T>
struct LogitPiece {
  static constexpr int kVec = 16 / sizeof(T);
  static constexpr int kRound = kLogitThreads * kVec;
  static constexpr int kRounds = sizeof(T) == 4 ? 4 : 2;
  static constexpr int kIds = kRound * kRounds;
  static constexpr int kList = 8192;               // list entries in shared memory
  static constexpr int kSmem = 8 * kIds + 4 * kList;
};

struct LogitsArgs {
  bc_logits_args a;
  int rounds;                 // of 16 bytes a thread per piece
  int pieces;                 // per row
  long long items, per_cta;   // pieces in all, and per CTA
};

__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// 16 bytes of logits with those whose bit is 0 at -inf
template <typename T>
__device__ __forceinline__ uint4 masked(uint4 w, uint32_t bits) {
  uint32_t x[4] = {w.x, w.y, w.z, w.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      if (!(bits >> i & 1u)) x[i] = 0xff800000u;
    } else {
      const uint32_t keep = (bits >> (2 * i) & 1u ? 0xffffu : 0u) | (bits >> (2 * i + 1) & 1u ? 0xffff0000u : 0u);
      x[i] = (x[i] & keep) | (0xff80ff80u & ~keep);
    }
  }
  return make_uint4(x[0], x[1], x[2], x[3]);
}

// Shared-memory atomics under a predicate, without a branch: most entries of a
// list are not of the piece at hand.
__device__ __forceinline__ void add_if(unsigned* p, unsigned x, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p red.shared.add.u32 [%0], %1;\n}" ::"r"(smem_addr(p)),
               "r"(x), "r"((unsigned)on) : "memory");
}
__device__ __forceinline__ void or_if(unsigned* p, unsigned x, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p red.shared.or.b32 [%0], %1;\n}" ::"r"(smem_addr(p)),
               "r"(x), "r"((unsigned)on) : "memory");
}
__device__ __forceinline__ void max_if(unsigned* p, unsigned x, bool on) {
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %2, 0;\n @p red.shared.max.u32 [%0], %1;\n}" ::"r"(smem_addr(p)),
               "r"(x), "r"((unsigned)on) : "memory");
}

__device__ __forceinline__ int clamp_at(int i, int hi) { return min(max(i, 0), hi); }

// the mask of row b, or null
__device__ __forceinline__ const uint32_t* mask_of(const bc_logits_args& a, int b) {
  if (!a.mask) return nullptr;
  const int m = a.mask_row ? a.mask_row[b] : b;
  return m >= 0 && m < a.n_masks ? a.mask + (size_t)m * ((a.vocab + 31) / 32) : nullptr;
}

template <typename T>
__global__ void __launch_bounds__(kLogitThreads, kLogitCtas) k_logits(const __grid_constant__ LogitsArgs g) {
  using P = LogitPiece<T>;
  constexpr int VEC = P::kVec;
  extern __shared__ __align__(16) uint8_t smem[];
  unsigned* s_mark = reinterpret_cast<unsigned*>(smem);               // [kIds] of the history
  unsigned* s_bias = s_mark + P::kIds;                                // [kIds] of the biases
  int* s_list = reinterpret_cast<int*>(s_bias + P::kIds);
  // [kList]: history, then biases, each padded to a multiple of 4
  const bc_logits_args& a = g.a;
  const int piece = g.rounds * P::kRound;
  const long long first = blockIdx.x * g.per_cta;
  int left = (int)min(g.per_cta, g.items - first);
  pdl_wait();
  pdl_trigger();
  if (left <= 0) return;

  // A piece of a row holds its ids from lo on, lo at a 16-byte boundary of the
  // logits (the first one begins up to VEC - 1 places before the row); those at
  // its places t0 .. t1 - 1 exist.
  struct Piece {
    int row, lo, t0, t1;
    const T* src;             // place 0 of it
    T* dst;
  };
  auto begin_row = [&](int row) {
    Piece x;
    x.row = row;
    x.src = static_cast<const T*>(a.logits) + (long long)row * a.stride;
    x.dst = static_cast<T*>(a.out) + (long long)row * a.out_stride;
    x.t0 = (int)(reinterpret_cast<uintptr_t>(x.src) % 16 / sizeof(T));
    x.lo = -x.t0;
    x.src -= x.t0;
    x.dst -= x.t0;
    x.t1 = min(piece, a.vocab - x.lo);
    return x;
  };
  auto move = [&](Piece& x, int by) {              // within the row
    x.lo += by;
    x.src += by;
    x.dst += by;
    x.t0 = 0;
    x.t1 = min(piece, a.vocab - x.lo);
  };
  auto fetch = [&](uint4 (&w)[P::kRounds], const Piece& x) {
    #pragma unroll
    for (int r = 0; r < P::kRounds; ++r) {
      const int t = r * P::kRound + VEC * threadIdx.x;
      if (t >= x.t0 && t + VEC <= x.t1) {
        w[r] = *reinterpret_cast<const uint4*>(x.src + t);
      } else if (t < x.t1 && t + VEC > x.t0) {
        T* y = reinterpret_cast<T*>(&w[r]);
        #pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (t + j >= x.t0 && t + j < x.t1) y[j] = x.src[t + j];
      }
    }
  };
  int p = (int)(first % g.pieces);
  Piece x = begin_row((int)(first / g.pieces));
  if (p) move(x, p * piece);
  uint4 w[P::kRounds], w_next[P::kRounds];
  fetch(w, x);
  for (int i = 4 * threadIdx.x; i < 2 * P::kIds; i += 4 * kLogitThreads)
    *reinterpret_cast<uint4*>(s_mark + i) = make_uint4(0, 0, 0, 0);

  int at_row = -1, h0 = 0, h1 = 0, b0 = 0, b1 = 0, nh = 0, nb = 0;   // nh, nb: entries in shared memory
  unsigned out0 = 0;
  float rep = 1.f, inv_rep = 1.f, freq = 0.f, pres = 0.f;
  const uint32_t* mask = nullptr;
  for (;;) {
    const bool more = --left > 0;
    if (x.row != at_row) {
      const int row = at_row = x.row;
      h0 = a.hist ? clamp_at(a.hist_start[row], a.n_hist) : 0;
      h1 = max(h0, a.hist ? clamp_at(a.hist_start[row + 1], a.n_hist) : 0);
      b0 = a.bias_ids ? clamp_at(a.bias_start[row], a.n_bias) : 0;
      b1 = max(b0, a.bias_ids ? clamp_at(a.bias_start[row + 1], a.n_bias) : 0);
      out0 = h0 + min(a.prompt_len ? max(a.prompt_len[row], 0) : 0, h1 - h0);       // behind the prompt
      rep = a.repetition ? a.repetition[row] : 1.f;
      // x / rep to within an ulp and a half, for one multiplication an id (41.1 us;
      // a division where the reciprocal is not a normal number: 42.9)
      inv_rep = __frcp_rn(rep);
      freq = a.frequency ? a.frequency[row] : 0.f;
      pres = a.presence ? a.presence[row] : 0.f;
      mask = mask_of(a, row);
      nh = min(h1 - h0, P::kList);
      const int pad = (nh + 3) & ~3;
      nb = min(b1 - b0, P::kList - pad);
      __syncthreads();                          // the list of the row before is done with
      // asynchronous copies: a thread's entries are all in flight at once
      auto bring = [&](const int* list, int count, int* to) {
        for (int i = threadIdx.x; i < count; i += kLogitThreads)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(to + i)), "l"(list + i) : "memory");
        if (threadIdx.x < (-count & 3)) to[count + threadIdx.x] = -1;
      };
      bring(a.hist + h0, nh, s_list);
      bring(a.bias_ids + b0, nb, s_list + pad);
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
    }
    const int v0 = x.lo + x.t0;
    const unsigned n = max(x.t1 - x.t0, 0);      // (a row's last piece may hold nothing)
    unsigned *mark0 = s_mark + x.t0, *bias0 = s_bias + x.t0;
    Piece next = x;                              // on its way until then
    if (more) {
      if (++p < g.pieces) {
        move(next, piece);
      } else {
        p = 0;
        next = begin_row(x.row + 1);
      }
      fetch(w_next, next);
    }
    uint32_t bits[P::kRounds];                   // on their way during the walks
    #pragma unroll
    for (int r = 0; r < P::kRounds; ++r) bits[r] = 0xffu;
    // The usual case: 16 bytes are of one word.  It is shifted where it is used,
    // so that nothing waits for it before the walks (44 against 47 us).
    const bool in_word = x.lo % 32 == 0;
    if (mask && in_word) {
      const uint32_t* m = mask + (x.lo >> 5);
      #pragma unroll
      for (int r = 0; r < P::kRounds; ++r) {
        const int t = r * P::kRound + VEC * threadIdx.x;
        if (t < x.t1) bits[r] = m[t >> 5];
      }
    } else if (mask) {
      #pragma unroll
      for (int r = 0; r < P::kRounds; ++r) {
        const int t = r * P::kRound + VEC * threadIdx.x;
        if (t >= x.t1 || t + VEC <= x.t0) continue;
        const int v = max(x.lo + t, 0), e = min(x.lo + t + VEC, a.vocab) - 1;    // first and last id of the 16 bytes
        const uint32_t m0 = mask[v >> 5], m1 = (e ^ v) >> 5 ? mask[e >> 5] : 0u;
        bits[r] = __funnelshift_r(m0, m1, v & 31) << (v - (x.lo + t));
      }
    }
    // use(i, ids - v0, step) for the entries of list[begin, stop), its first
    // `held` entries at s_list[from]; four at a time: entries i, i + step, ..
    auto walk = [&](const int* list, int begin, int stop, int from, int held, auto use) {
      for (int i = 4 * threadIdx.x; i < held; i += 4 * kLogitThreads) {
        const int4 id = *reinterpret_cast<const int4*>(s_list + from + i);
        const unsigned v[4] = {(unsigned)id.x - (unsigned)v0, (unsigned)id.y - (unsigned)v0, (unsigned)id.z - (unsigned)v0,
                               (unsigned)id.w - (unsigned)v0};
        use((unsigned)(begin + i), v, 1u);
      }
      for (unsigned i0 = begin + held + threadIdx.x; i0 < (unsigned)stop; i0 += kLogitWalk * kLogitThreads) {
        unsigned v[kLogitWalk];
        #pragma unroll
        for (int j = 0; j < kLogitWalk; ++j) {
          const unsigned i = i0 + j * kLogitThreads;
          v[j] = i < (unsigned)stop ? (unsigned)list[i] - (unsigned)v0 : 0xffffffffu;
        }
        #pragma unroll
        for (int j = 0; j < kLogitWalk; j += 4) use(i0 + j * kLogitThreads, v + j, (unsigned)kLogitThreads);
      }
    };
    const bool listed = h1 > h0 || b1 > b0;
    if (listed) {
      walk(a.hist, h0, h1, 0, nh, [&](unsigned i, const unsigned* v, unsigned step) {
        if (i >= out0) {
          #pragma unroll
          for (int j = 0; j < 4; ++j) add_if(mark0 + v[j], 1u, v[j] < n);
        } else if (i + 3 * step < out0) {
          #pragma unroll
          for (int j = 0; j < 4; ++j) or_if(mark0 + v[j], 0x80000000u, v[j] < n);
        } else {
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool prompt = i + j * step < out0;
            or_if(mark0 + v[j], 0x80000000u, prompt && v[j] < n);
            add_if(mark0 + v[j], 1u, !prompt && v[j] < n);
          }
        }
      });
      walk(a.bias_ids, b0, b1, (nh + 3) & ~3, nb, [&](unsigned i, const unsigned* v, unsigned step) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) max_if(bias0 + v[j], i + j * step - b0 + 1, v[j] < n);
      });
      __syncthreads();
    }
    // the marked ids among the 16 bytes at place t, whose words are cleared;
    // four at a time without branches, since most warps find some of a long
    // history (42 against 44 us)
    auto change = [&](uint4& at_t, int t) {
      T* y = reinterpret_cast<T*>(&at_t);
      #pragma unroll
      for (int q = 0; q < VEC; q += 4) {
        uint4* mark = reinterpret_cast<uint4*>(s_mark + t + q);
        uint4* bias = reinterpret_cast<uint4*>(s_bias + t + q);
        const uint4 c4 = *mark, w4 = b1 > b0 ? *bias : make_uint4(0, 0, 0, 0);
        if (!(c4.x | c4.y | c4.z | c4.w | w4.x | w4.y | w4.z | w4.w)) continue;
        *mark = *bias = make_uint4(0, 0, 0, 0);
        const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w}, at[4] = {w4.x, w4.y, w4.z, w4.w};
        float z[4];
        #pragma unroll
        for (int j = 0; j < 4; ++j) {
          const unsigned outputs = c[j] & 0x7fffffffu;
          const float u = value_of(y[q + j]), f = u > 0.f ? inv_rep : rep;
          const float off = outputs ? __fmul_rn(freq, (float)outputs) + pres : 0.f;
          z[j] = c[j] ? __fmul_rn(u, f) - off : u;
        }
        if (w4.x | w4.y | w4.z | w4.w) {
          #pragma unroll
          for (int j = 0; j < 4; ++j)
            if (at[j]) z[j] += a.bias_vals[b0 + at[j] - 1];
        }
        #pragma unroll
        for (int j = 0; j < 4; ++j) store_one(y + q + j, z[j]);
      }
    };
    const bool wide = reinterpret_cast<uintptr_t>(x.dst) % 16 == 0;
    #pragma unroll
    for (int r = 0; r < P::kRounds; ++r) {
      const int t = r * P::kRound + VEC * threadIdx.x;
      if (t >= x.t1 || t + VEC <= x.t0) continue;
      if (listed) change(w[r], t);
      if (mask) w[r] = masked<T>(w[r], bits[r] >> (in_word ? t & 31 : 0));
      if (wide && t >= x.t0 && t + VEC <= x.t1) {
        *reinterpret_cast<uint4*>(x.dst + t) = w[r];
      } else {
        const T* y = reinterpret_cast<const T*>(&w[r]);
        #pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (t + j >= x.t0 && t + j < x.t1) x.dst[t + j] = y[j];
      }
    }
    if (!more) break;
    if (listed) __syncthreads();                 // the marks are clear
    x = next;
    #pragma unroll
    for (int r = 0; r < P::kRounds; ++r) w[r] = w_next[r];
  }
}

}  // namespace bc

using namespace bc;

template <typename T>
static cudaError_t launch_logits(const LogitsArgs& g, dim3 grid, cudaStream_t st) {
  constexpr int smem = LogitPiece<T>::kSmem;
  static std::atomic<unsigned long long> ready{0};     // once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load() >> dev & 1))) {
    e = cudaFuncSetAttribute(k_logits<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) ready.fetch_or(1ull << dev);
  }
  return e != cudaSuccess ? e : launch_op(k_logits<T>, grid, dim3(kLogitThreads), smem, st, g);
}

extern "C" bc_status bc_logits_adjust(const bc_logits_args* a, void* stream) {
  const char* who = "bc_logits_adjust";
  if (!a) return entry_fail(BC_EINVAL, "%s: null arguments", who);
  if (!a->logits || !a->out) return entry_fail(BC_EINVAL, "%s: null pointer", who);
  if (a->dtype != BC_F32 && a->dtype != BC_BF16) return entry_fail(BC_EINVAL, "%s: bad dtype %d", who, (int)a->dtype);
  if (a->batch < 1 || a->batch > 65535) return entry_fail(BC_EINVAL, "%s: batch %d outside [1, 65535]", who, a->batch);
  if (a->vocab < 1 || a->vocab > INT32_MAX - 32768) return entry_fail(BC_EINVAL, "%s: bad vocab %d", who, a->vocab);
  if (a->stride < a->vocab || a->out_stride < a->vocab)
    return entry_fail(BC_EINVAL, "%s: strides must be at least vocab", who);
  if (a->out == a->logits && a->out_stride != a->stride)
    return entry_fail(BC_EINVAL, "%s: an update in place needs equal strides", who);
  const size_t es = a->dtype == BC_F32 ? 4 : 2;
  if (!aligned(a->logits, es) || !aligned(a->out, es))
    return entry_fail(BC_EINVAL, "%s: logits and out must be aligned to their type", who);
  if (a->hist && (!a->hist_start || a->n_hist < 0)) return entry_fail(BC_EINVAL, "%s: hist needs hist_start and n_hist", who);
  if (a->bias_ids && (!a->bias_vals || !a->bias_start || a->n_bias < 0))
    return entry_fail(BC_EINVAL, "%s: bias_ids needs bias_vals, bias_start and n_bias", who);
  if (a->mask && a->n_masks < (a->mask_row ? 0 : a->batch))
    return entry_fail(BC_EINVAL, "%s: n_masks must cover the batch without mask_row", who);
  LogitsArgs g{*a, 1, 0, 0, 0};
  constexpr int kCtas = 148 * kLogitCtas;
  const bool f32 = a->dtype == BC_F32;
  const int vec = f32 ? LogitPiece<float>::kVec : LogitPiece<__nv_bfloat16>::kVec;
  const int round = kLogitThreads * vec, most = f32 ? LogitPiece<float>::kRounds : LogitPiece<__nv_bfloat16>::kRounds;
  // the rounds that take least, at one more per piece for the walks: fewer
  // where a CTA would get a second piece for want of others (16 rows 7.8 us)
  long long best = 0;
  for (int r = 1; r <= most; ++r) {
    // (a row may begin off a boundary)
    const long long pieces = (a->vocab + (long long)(vec - 1) + r * round - 1) / (r * round);
    const long long cost = (a->batch * pieces + kCtas - 1) / kCtas * (r + 1);
    if (r > 1 && cost > best) continue;
    best = cost;
    g.rounds = r;
    g.pieces = (int)pieces;
  }
  g.items = (long long)a->batch * g.pieces;
  const long long ctas = std::min<long long>(g.items, kCtas);
  g.per_cta = (g.items + ctas - 1) / ctas;
  const dim3 grid((unsigned)((g.items + g.per_cta - 1) / g.per_cta));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return entry_cuda(f32 ? launch_logits<float>(g, grid, st) : launch_logits<__nv_bfloat16>(g, grid, st),
                    who);
}
