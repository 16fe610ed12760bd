// Penalties, biases and grammar masks on logits (bc_logits_adjust): one pass
// over the logits, HBM-bound.
//
// Persistent CTAs take pieces of 2048 to 8192 ids, neighbours of a row one
// after the other, and load a piece's logits (4 a thread and round) while the
// one before is worked on.  A row's history and biases are read once per row
// and CTA into shared memory.  For each piece the CTA walks them and marks the
// ids that fall into the piece, a word per id and list; each thread then looks
// its own ids up and clears their words.  A word of the history is bit 31,
// "seen in the prompt", and the count of the output tokens; a word of the
// biases the place of the last entry for the id (a maximum), so no result
// depends on the order of the atomics.
// 160 rows of 128256 f32 logits with histories of up to 8192 tokens, 32 biases
// and masks take 46 us (3.5 TB/s of logits; 29 us without lists, the copy's
// rate); 68 us with a CTA a piece that walks the lists in L2, 55 us as a copy
// and a scatter from hash tables.  The walks' instructions bound the rest.
#include "common.cuh"
#include "entry.h"

#include <algorithm>
#include <atomic>

namespace bc {

constexpr int kLogitThreads = 512;
constexpr int kLogitRound = 4 * kLogitThreads;   // ids per round
constexpr int kLogitRounds = 4;                  // at most, per piece
constexpr int kLogitCtas = 2;                    // per SM
constexpr int kLogitList = 8192;                 // list entries in shared memory
constexpr int kLogitWalk = 8;                    // further ones per thread in flight

struct LogitsArgs {
  bc_logits_args a;
  int rounds;                 // of kLogitRound ids per piece
  int pieces;                 // per row
  long long items, per_cta;   // pieces in all, and per CTA
};

__device__ __forceinline__ float4 load_four(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load_four(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void store_four(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store_four(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}
__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_one(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

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
  extern __shared__ __align__(16) unsigned s_mark[];            // [kLogitRounds * kLogitRound]
  unsigned* s_bias = s_mark + kLogitRounds * kLogitRound;       // the same for the biases
  int* s_list = reinterpret_cast<int*>(s_bias + kLogitRounds * kLogitRound);
  // [kLogitList]: history, then biases, each padded to a multiple of 4
  const bc_logits_args& a = g.a;
  const int piece = g.rounds * kLogitRound;
  const long long first = blockIdx.x * g.per_cta;
  int left = (int)min(g.per_cta, g.items - first);
  pdl_wait();
  pdl_trigger();
  if (left <= 0) return;

  int row = (int)(first / g.pieces), v0 = (int)(first % g.pieces) * piece;
  // rows of any alignment: four at a time where both sides allow it
  auto load = [&](float (&x)[kLogitRounds][4], int r, int v) {
    const T* src = static_cast<const T*>(a.logits) + (long long)r * a.stride + v;
    const int n = min(piece, a.vocab - v);
    const bool wide = (reinterpret_cast<uintptr_t>(src) & (4 * sizeof(T) - 1)) == 0;
    #pragma unroll
    for (int k = 0; k < kLogitRounds; ++k) {
      const int i = k * kLogitRound + 4 * threadIdx.x;
      if (wide && i + 4 <= n) {
        const float4 y = load_four(src + i);
        x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
      } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j) x[k][j] = i + j < n ? value_of(src[i + j]) : 0.f;
      }
    }
  };
  float x[kLogitRounds][4], next[kLogitRounds][4];
  load(x, row, v0);
  #pragma unroll
  for (int k = 0; k < 2 * kLogitRounds; ++k)
    *reinterpret_cast<uint4*>(s_mark + k * kLogitRound + 4 * threadIdx.x) = make_uint4(0, 0, 0, 0);

  int at_row = -1, h0 = 0, h1 = 0, b0 = 0, b1 = 0, nh = 0, nb = 0;   // nh, nb: entries in shared memory
  unsigned out0 = 0;
  float rep = 1.f, inv_rep = 1.f, freq = 0.f, pres = 0.f;
  const uint32_t* mask = nullptr;
  for (;;) {
    const bool more = --left > 0;
    const int next_row = v0 + piece < a.vocab ? row : row + 1, next_v0 = v0 + piece < a.vocab ? v0 + piece : 0;
    if (more) load(next, next_row, next_v0);
    if (row != at_row) {
      at_row = row;
      h0 = a.hist ? clamp_at(a.hist_start[row], a.n_hist) : 0;
      h1 = max(h0, a.hist ? clamp_at(a.hist_start[row + 1], a.n_hist) : 0);
      b0 = a.bias_ids ? clamp_at(a.bias_start[row], a.n_bias) : 0;
      b1 = max(b0, a.bias_ids ? clamp_at(a.bias_start[row + 1], a.n_bias) : 0);
      out0 = h0 + min(a.prompt_len ? max(a.prompt_len[row], 0) : 0, h1 - h0);       // behind the prompt
      rep = a.repetition ? a.repetition[row] : 1.f;
      inv_rep = __frcp_rn(rep);                 // x / rep to within an ulp and a half, for one multiplication an id
      freq = a.frequency ? a.frequency[row] : 0.f;
      pres = a.presence ? a.presence[row] : 0.f;
      mask = mask_of(a, row);
      nh = min(h1 - h0, kLogitList);
      const int pad = (nh + 3) & ~3;
      nb = min(b1 - b0, kLogitList - pad);
      __syncthreads();                          // the list of the row before is done with
      // asynchronous copies: a thread's entries are all in flight at once
      auto fetch = [&](const int* list, int count, int* to) {
        for (int i = threadIdx.x; i < count; i += kLogitThreads)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(to + i)), "l"(list + i) : "memory");
        if (threadIdx.x < (-count & 3)) to[count + threadIdx.x] = -1;
      };
      fetch(a.hist + h0, nh, s_list);
      fetch(a.bias_ids + b0, nb, s_list + pad);
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
    }
    const int n = min(piece, a.vocab - v0);
    uint32_t bits[kLogitRounds];                 // on their way during the walks
    #pragma unroll
    for (int k = 0; k < kLogitRounds; ++k) {
      const int i = k * kLogitRound + 4 * threadIdx.x;
      bits[k] = mask && i < n ? mask[(v0 + i) >> 5] >> (i & 31) : 0xfu;
    }
    // mark(i, ids - v0, step) for the entries of
    // list[begin, stop), its first `held` entries at s_list[from]; four at a
    // time: entries i, i + step, ..
    auto walk = [&](const int* list, int begin, int stop, int from, int held, auto mark) {
      for (int i = 4 * threadIdx.x; i < held; i += kLogitRound) {
        const int4 id = *reinterpret_cast<const int4*>(s_list + from + i);
        const unsigned v[4] = {(unsigned)id.x - (unsigned)v0, (unsigned)id.y - (unsigned)v0, (unsigned)id.z - (unsigned)v0,
                               (unsigned)id.w - (unsigned)v0};
        mark((unsigned)(begin + i), v, 1u);
      }
      for (unsigned i0 = begin + held + threadIdx.x; i0 < (unsigned)stop; i0 += kLogitWalk * kLogitThreads) {
        unsigned v[kLogitWalk];
        #pragma unroll
        for (int j = 0; j < kLogitWalk; ++j) {
          const unsigned i = i0 + j * kLogitThreads;
          v[j] = i < (unsigned)stop ? (unsigned)list[i] - (unsigned)v0 : 0xffffffffu;
        }
        #pragma unroll
        for (int j = 0; j < kLogitWalk; j += 4) mark(i0 + j * kLogitThreads, v + j, (unsigned)kLogitThreads);
      }
    };
    if (h1 > h0) {
      walk(a.hist, h0, h1, 0, nh, [&](unsigned i, const unsigned* v, unsigned step) {
        if (i >= out0) {
          #pragma unroll
          for (int j = 0; j < 4; ++j) add_if(s_mark + v[j], 1u, v[j] < (unsigned)n);
        } else {
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            const bool prompt = i + j * step < out0;
            or_if(s_mark + v[j], 0x80000000u, prompt && v[j] < (unsigned)n);
            add_if(s_mark + v[j], 1u, !prompt && v[j] < (unsigned)n);
          }
        }
      });
    }
    if (b1 > b0) {
      walk(a.bias_ids, b0, b1, (nh + 3) & ~3, nb,
           [&](unsigned i, const unsigned* v, unsigned step) {
             #pragma unroll
             for (int j = 0; j < 4; ++j) max_if(s_bias + v[j], i + j * step - b0 + 1, v[j] < (unsigned)n);
           });
    }
    if (h1 > h0 || b1 > b0) {
      __syncthreads();
      // the thread's marked ids, whose words are cleared
      #pragma unroll
      for (int k = 0; k < kLogitRounds; ++k) {
        const int i = k * kLogitRound + 4 * threadIdx.x;
        if (i >= n) break;
        const uint4 c4 = *reinterpret_cast<const uint4*>(s_mark + i);
        if (c4.x | c4.y | c4.z | c4.w) {
          *reinterpret_cast<uint4*>(s_mark + i) = make_uint4(0, 0, 0, 0);
          const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w};
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (!c[j]) continue;
            x[k][j] *= x[k][j] > 0.f ? inv_rep : rep;
            if (c[j] & 0x7fffffffu) x[k][j] -= __fmul_rn(freq, (float)(c[j] & 0x7fffffffu)) + pres;
          }
        }
        if (b1 == b0) continue;
        const uint4 w4 = *reinterpret_cast<const uint4*>(s_bias + i);
        if (w4.x | w4.y | w4.z | w4.w) {
          *reinterpret_cast<uint4*>(s_bias + i) = make_uint4(0, 0, 0, 0);
          const unsigned w[4] = {w4.x, w4.y, w4.z, w4.w};
          #pragma unroll
          for (int j = 0; j < 4; ++j)
            if (w[j]) x[k][j] += a.bias_vals[b0 + w[j] - 1];
        }
      }
      __syncthreads();
    }
    T* dst = static_cast<T*>(a.out) + (long long)row * a.out_stride + v0;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & (4 * sizeof(T) - 1)) == 0;
    #pragma unroll
    for (int k = 0; k < kLogitRounds; ++k) {
      const int i = k * kLogitRound + 4 * threadIdx.x;
      if (i >= n) break;
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        if (!(bits[k] >> j & 1u)) x[k][j] = -INFINITY;
      if (wide && i + 4 <= n) {
        store_four(dst + i, make_float4(x[k][0], x[k][1], x[k][2], x[k][3]));
      } else {
        #pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < n) store_one(dst + i + j, x[k][j]);
      }
    }
    if (!more) break;
    row = next_row;
    v0 = next_v0;
    #pragma unroll
    for (int k = 0; k < kLogitRounds; ++k)
      #pragma unroll
      for (int j = 0; j < 4; ++j) x[k][j] = next[k][j];
  }
}

}  // namespace bc

using namespace bc;

template <typename T>
static cudaError_t launch_logits(const LogitsArgs& g, dim3 grid, cudaStream_t st) {
  constexpr int smem = 4 * (2 * kLogitRounds * kLogitRound + kLogitList);
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
  // pieces no smaller than give every CTA one: each walks the lists
  const long long per = (long long)kCtas * kLogitRound;
  g.rounds = (int)std::min<long long>(kLogitRounds, ((long long)a->batch * a->vocab + per - 1) / per);
  const int piece = g.rounds * kLogitRound;
  g.pieces = (int)((a->vocab + (long long)piece - 1) / piece);
  g.items = (long long)a->batch * g.pieces;
  const long long ctas = std::min<long long>(g.items, kCtas);
  g.per_cta = (g.items + ctas - 1) / ctas;
  const dim3 grid((unsigned)((g.items + g.per_cta - 1) / g.per_cta));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return entry_cuda(a->dtype == BC_F32 ? launch_logits<float>(g, grid, st) : launch_logits<__nv_bfloat16>(g, grid, st),
                    who);
}
