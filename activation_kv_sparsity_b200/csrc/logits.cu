// Penalties, biases and grammar masks on logits (bc_logits_adjust): one pass
// over the logits.
//
// A CTA owns a piece of one row's vocabulary, 1 to 8 times 1024 ids.  It
// starts to load its logits (4 a thread and round), clears a word per id in
// shared memory, walks the row's history (and its biases) and keeps what
// falls into its piece: bit 31 of the word is "seen", the rest counts the
// tokens behind the prompt; a second word holds the place of the last bias
// listed for the id (a maximum, so the result does not depend on order).
// Then the logits go through.  Counters in shared memory instead of a table
// in HBM cost a walk of the history per piece, from L2 and 1/8 to 1/16 of the
// logits' bytes for histories of thousands of tokens.
#include "common.cuh"
#include "entry.h"

#include <algorithm>
#include <atomic>

namespace bc {

constexpr int kLogitThreads = 256;
constexpr int kLogitRound = 4 * kLogitThreads;   // ids per round
constexpr int kLogitRounds = 8;                  // at most, per CTA

struct LogitsArgs {
  bc_logits_args a;
  int rounds;       // of kLogitRound ids per CTA
};

// four logits as loaded, and their values
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 x;
  __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void set(int i, float v) { (&x.x)[i] = v; }
  __device__ __forceinline__ float get(int i) const { return (&x.x)[i]; }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = x; }
  static __device__ __forceinline__ float value(float v) { return v; }
  static __device__ __forceinline__ float round(float v) { return v; }
};
template <>
struct Four<__nv_bfloat16> {
  uint2 x;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void set(int i, __nv_bfloat16 v) {
    uint32_t& w = i < 2 ? x.x : x.y;
    const uint32_t u = __bfloat16_as_ushort(v);
    w = i & 1 ? (w & 0xffffu) | (u << 16) : (w & 0xffff0000u) | u;
  }
  __device__ __forceinline__ __nv_bfloat16 get(int i) const {
    const uint32_t w = i < 2 ? x.x : x.y;
    return __ushort_as_bfloat16((unsigned short)(i & 1 ? w >> 16 : w & 0xffffu));
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = x; }
  static __device__ __forceinline__ float value(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 round(float v) { return __float2bfloat16_rn(v); }
};

template <typename T>
__global__ void __launch_bounds__(kLogitThreads) k_logits(const __grid_constant__ LogitsArgs g) {
  extern __shared__ __align__(16) unsigned s_count[];
  const bc_logits_args& a = g.a;
  const int piece = g.rounds * kLogitRound;
  const int b = blockIdx.y, v0 = blockIdx.x * piece, n = min(piece, a.vocab - v0);
  unsigned* s_bias = s_count + piece;        // place of the last bias + 1
  pdl_wait();
  pdl_trigger();
  const T* src = static_cast<const T*>(a.logits) + (long long)b * a.stride + v0;
  T* dst = static_cast<T*>(a.out) + (long long)b * a.out_stride + v0;
  // rows of any alignment: four at a time where both sides allow it
  const bool wide = ((reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst)) & (4 * sizeof(T) - 1)) == 0;
  Four<T> x[kLogitRounds];
  #pragma unroll
  for (int r = 0; r < kLogitRounds; ++r) {
    const int i = r * kLogitRound + 4 * threadIdx.x;
    if (wide && i + 4 <= n) {
      x[r].load(src + i);
    } else {
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) x[r].set(j, src[i + j]);
    }
  }
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_row ? a.mask_row[b] : b;
    if (m >= 0 && m < a.n_masks) mask = a.mask + (size_t)m * ((a.vocab + 31) / 32) + v0 / 32;
  }
  auto clamp_at = [](int i, int hi) { return min(max(i, 0), hi); };
  const int h0 = a.hist ? clamp_at(a.hist_start[b], a.n_hist) : 0;
  const int h1 = a.hist ? clamp_at(a.hist_start[b + 1], a.n_hist) : 0;
  const int b0 = a.bias_ids ? clamp_at(a.bias_start[b], a.n_bias) : 0;
  const int b1 = a.bias_ids ? clamp_at(a.bias_start[b + 1], a.n_bias) : 0;
  const int h_out = h0 + min(a.prompt_len ? max(a.prompt_len[b], 0) : 0, max(h1 - h0, 0));   // first output token
  if (h1 > h0)
    for (int i = threadIdx.x; i < piece / 4; i += kLogitThreads)
      reinterpret_cast<uint4*>(s_count)[i] = make_uint4(0, 0, 0, 0);
  if (b1 > b0)
    for (int i = threadIdx.x; i < piece / 4; i += kLogitThreads)
      reinterpret_cast<uint4*>(s_bias)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (unsigned i0 = h0 + threadIdx.x; i0 < (unsigned)h1; i0 += kLogitRound) {
    unsigned v[4];
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      const unsigned i = i0 + j * kLogitThreads;
      v[j] = i < (unsigned)h1 ? (unsigned)a.hist[i] - (unsigned)v0 : 0xffffffffu;
    }
    #pragma unroll
    for (int j = 0; j < 4; ++j)
      if (v[j] < (unsigned)n) {
        if (i0 + j * kLogitThreads >= (unsigned)h_out) atomicAdd(&s_count[v[j]], 1u);
        atomicOr(&s_count[v[j]], 0x80000000u);
      }
  }
  for (unsigned i = b0 + threadIdx.x; i < (unsigned)b1; i += kLogitThreads) {
    const unsigned v = (unsigned)a.bias_ids[i] - (unsigned)v0;
    if (v < (unsigned)n) atomicMax(&s_bias[v], i - b0 + 1);
  }
  __syncthreads();
  #pragma unroll
  for (int r = 0; r < kLogitRounds; ++r) {
    const int i = r * kLogitRound + 4 * threadIdx.x;
    if (i >= n) break;
    const uint4 c4 = h1 > h0 ? *reinterpret_cast<const uint4*>(s_count + i) : make_uint4(0, 0, 0, 0);
    const uint4 w4 = b1 > b0 ? *reinterpret_cast<const uint4*>(s_bias + i) : make_uint4(0, 0, 0, 0);
    const uint32_t bits = mask ? mask[i >> 5] >> (i & 31) : 0xfu;
    const unsigned c[4] = {c4.x, c4.y, c4.z, c4.w}, w[4] = {w4.x, w4.y, w4.z, w4.w};
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y = Four<T>::value(x[r].get(j));
      if (c[j]) {
        if (a.repetition) y = y > 0.f ? __fdiv_rn(y, rep) : y * rep;
        if (c[j] & 0x7fffffffu) y -= __fmul_rn(freq, (float)(c[j] & 0x7fffffffu)) + pres;
      }
      if (w[j]) y += a.bias_vals[b0 + w[j] - 1];
      if (!(bits >> j & 1u)) y = -INFINITY;
      if (c[j] || w[j] || !(bits >> j & 1u)) x[r].set(j, Four<T>::round(y));
    }
    if (wide && i + 4 <= n) {
      x[r].store(dst + i);
    } else {
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) dst[i + j] = x[r].get(j);
    }
  }
}

}  // namespace bc

using namespace bc;

template <typename T>
static cudaError_t launch_logits(const LogitsArgs& g, dim3 grid, size_t smem, cudaStream_t st) {
  // once per device: room for the largest piece
  static std::atomic<unsigned long long> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev >= 64 || !(ready.load() >> dev & 1))) {
    e = cudaFuncSetAttribute(k_logits<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, 8 * kLogitRounds * kLogitRound);
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
  LogitsArgs g{*a, 1};
  // pieces as large as leave 6 CTAs an SM: fewer walks of the histories
  const long long all = (long long)a->batch * a->vocab;
  g.rounds = (int)std::min<long long>(kLogitRounds, std::max<long long>(1, all / (148LL * 6 * kLogitRound)));
  const int piece = g.rounds * kLogitRound;
  const dim3 grid((unsigned)((a->vocab + (long long)piece - 1) / piece), a->batch);
  const size_t smem = a->bias_ids ? 8ull * piece : a->hist ? 4ull * piece : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return entry_cuda(a->dtype == BC_F32 ? launch_logits<float>(g, grid, smem, st)
                                       : launch_logits<__nv_bfloat16>(g, grid, smem, st), who);
}
