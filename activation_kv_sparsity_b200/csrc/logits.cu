// Penalties, biases and grammar masks on logits (bc_logits_adjust): one pass
// over the logits.
//
// A CTA owns a piece of one row's vocabulary.  It clears a word per token id
// in shared memory, walks the row's history (and its biases) and keeps what
// falls into its piece: bit 31 of the word is "seen", the rest counts the
// tokens behind the prompt; a second word holds the place of the last bias
// listed for the id (a maximum, so the result does not depend on order).
// Then it streams the logits through.
#include "common.cuh"
#include "entry.h"

#include <algorithm>

namespace bc {

constexpr int kLogitThreads = 256;

struct LogitsArgs {
  bc_logits_args a;
  int piece;        // token ids per CTA (a multiple of 32)
};

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

template <typename T>
__global__ void __launch_bounds__(kLogitThreads) k_logits(LogitsArgs g) {
  extern __shared__ unsigned s_count[];
  const bc_logits_args& a = g.a;
  const int b = blockIdx.y, v0 = blockIdx.x * g.piece, n = min(g.piece, a.vocab - v0);
  unsigned* s_bias = s_count + g.piece;      // place of the last bias + 1
  pdl_wait();
  pdl_trigger();
  auto clamp_at = [](int x, int hi) { return min(max(x, 0), hi); };
  if (a.hist)
    for (int i = threadIdx.x; i < n; i += kLogitThreads) s_count[i] = 0u;
  if (a.bias_ids)
    for (int i = threadIdx.x; i < n; i += kLogitThreads) s_bias[i] = 0u;
  __syncthreads();
  int bias0 = 0;
  if (a.hist) {
    const int h0 = clamp_at(a.hist_start[b], a.n_hist), h1 = clamp_at(a.hist_start[b + 1], a.n_hist);
    const int pl = a.prompt_len ? max(a.prompt_len[b], 0) : 0;
    for (int i = h0 + threadIdx.x; i < h1; i += kLogitThreads) {
      const unsigned v = (unsigned)a.hist[i] - (unsigned)v0;
      if (v < (unsigned)n) {
        if (i - h0 >= pl) atomicAdd(&s_count[v], 1u);
        atomicOr(&s_count[v], 0x80000000u);
      }
    }
  }
  if (a.bias_ids) {
    bias0 = clamp_at(a.bias_start[b], a.n_bias);
    const int b1 = clamp_at(a.bias_start[b + 1], a.n_bias);
    for (int i = bias0 + threadIdx.x; i < b1; i += kLogitThreads) {
      const unsigned v = (unsigned)a.bias_ids[i] - (unsigned)v0;
      if (v < (unsigned)n) atomicMax(&s_bias[v], (unsigned)(i - bias0 + 1));
    }
  }
  __syncthreads();
  const float rep = a.repetition ? a.repetition[b] : 1.f;
  const float freq = a.frequency ? a.frequency[b] : 0.f;
  const float pres = a.presence ? a.presence[b] : 0.f;
  const uint32_t* mask = nullptr;
  if (a.mask) {
    const int m = a.mask_row ? a.mask_row[b] : b;
    if (m >= 0 && m < a.n_masks) mask = a.mask + (size_t)m * ((a.vocab + 31) / 32);
  }
  const T* src = static_cast<const T*>(a.logits) + (long long)b * a.stride + v0;
  T* dst = static_cast<T*>(a.out) + (long long)b * a.out_stride + v0;
  for (int i = threadIdx.x; i < n; i += kLogitThreads) {
    float x = to_f<T>(src[i]);
    const unsigned c = a.hist ? s_count[i] : 0u;
    if (c) {
      if (a.repetition) x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      if (c & 0x7fffffffu) x -= __fmul_rn(freq, (float)(c & 0x7fffffffu)) + pres;
    }
    if (a.bias_ids && s_bias[i]) x += a.bias_vals[bias0 + s_bias[i] - 1];
    if (mask && !((mask[(v0 + i) >> 5] >> ((v0 + i) & 31)) & 1u)) x = -INFINITY;
    from_f(x, dst + i);
  }
}

}  // namespace bc

using namespace bc;

extern "C" bc_status bc_logits_adjust(const bc_logits_args* a, void* stream) {
  const char* who = "bc_logits_adjust";
  if (!a) return entry_fail(BC_EINVAL, "%s: null arguments", who);
  if (!a->logits || !a->out) return entry_fail(BC_EINVAL, "%s: null pointer", who);
  if (a->dtype != BC_F32 && a->dtype != BC_BF16) return entry_fail(BC_EINVAL, "%s: bad dtype %d", who, (int)a->dtype);
  if (a->batch < 1 || a->batch > 65535) return entry_fail(BC_EINVAL, "%s: batch %d outside [1, 65535]", who, a->batch);
  if (a->vocab < 1 || a->vocab > INT32_MAX - 32768) return entry_fail(BC_EINVAL, "%s: bad vocab %d", who, a->vocab);
  if (a->stride < a->vocab || a->out_stride < a->vocab)
    return entry_fail(BC_EINVAL, "%s: strides must be at least vocab", who);
  const size_t es = a->dtype == BC_F32 ? 4 : 2;
  if (!aligned(a->logits, es) || !aligned(a->out, es))
    return entry_fail(BC_EINVAL, "%s: logits and out must be aligned to their type", who);
  if (a->hist && (!a->hist_start || a->n_hist < 0)) return entry_fail(BC_EINVAL, "%s: hist needs hist_start and n_hist", who);
  if (a->bias_ids && (!a->bias_vals || !a->bias_start || a->n_bias < 0))
    return entry_fail(BC_EINVAL, "%s: bias_ids needs bias_vals, bias_start and n_bias", who);
  if (a->mask && a->n_masks < (a->mask_row ? 0 : a->batch))
    return entry_fail(BC_EINVAL, "%s: n_masks must cover the batch without mask_row", who);
  LogitsArgs g{*a, 0};
  g.piece = std::min(4096, (a->vocab + 31) / 32 * 32);
  const dim3 grid((a->vocab + g.piece - 1) / g.piece, a->batch);
  const size_t smem = 8ull * g.piece;
  cudaError_t e = a->dtype == BC_F32
                      ? launch_op(k_logits<float>, grid, dim3(kLogitThreads), smem, static_cast<cudaStream_t>(stream), g)
                      : launch_op(k_logits<__nv_bfloat16>, grid, dim3(kLogitThreads), smem,
                                  static_cast<cudaStream_t>(stream), g);
  return entry_cuda(e, who);
}
