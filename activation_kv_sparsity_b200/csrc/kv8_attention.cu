// Attention of a ragged batch over the 8-bit paged cache (bc_kv8_attention).
//
//   x_t = scale q.k_t, capped and biased as asked;  o = sum_t p_t v_t,
//   p = softmax(x) over the tokens the row sees,
// in one pass: running maximum m and sum l in base 2, o rescaled as m grows.
#include "entry.h"
#include "kv8.cuh"

#include <algorithm>

namespace bc {

constexpr int kKv8AttnWarps = 4;

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return min(max(x, lo), hi); }

// A CTA takes one query row of one query head; its warps share the pages.
template <int HD, int TYPE, typename T>
__global__ void __launch_bounds__(kKv8AttnWarps * 32) k_kv8_attn(bc_kv8_attention_args a) {
  constexpr int DPL = HD / 32;      // dims per lane
  __shared__ float s_o[kKv8AttnWarps][HD];
  __shared__ float s_m[kKv8AttnWarps], s_l[kKv8AttnWarps];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.y / a.max_q, i = blockIdx.y % a.max_q, j = blockIdx.x, h = j / a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = (int)min((long long)max(a.lens[b], 0), (long long)a.max_blocks * kPage);
  const int r0 = a.q_start ? a.q_start[b] : b, n_own = a.q_start ? a.q_start[b + 1] - r0 : 1;
  const long long row = (long long)r0 + i;
  if (i >= n_own || row < 0 || row >= a.n_q) return;
  const long long p = (long long)n - n_own + i;
  const T* q = static_cast<const T*>(a.q) + row * a.q_stride + (long long)j * HD + lane * DPL;
  float qv[DPL], o[DPL];
  #pragma unroll
  for (int d = 0; d < DPL; ++d) {
    qv[d] = (float)q[d];
    o[d] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const float slope = a.slopes ? a.slopes[j] : 0.f;
  const int n_blk = (n + kPage - 1) / kPage;
  const int* list = a.pages ? a.pages + ((long long)b * a.n_kv_heads + h) * a.max_sel : nullptr;
  const int count = list ? clampi(a.n_sel[b], 0, a.max_sel) : n_blk;
  for (int e = warp; e < count; e += kKv8AttnWarps) {
    const int lp = list ? list[e] : e;
    if (lp < 0 || lp >= n_blk) continue;
    const int page = a.table[(long long)b * a.max_blocks + lp];
    if (page < 0 || page >= a.n_pages) continue;
    const uint8_t* blk = static_cast<const uint8_t*>(a.pool) +
                         ((long long)page * a.n_kv_heads + h) * kv8_block_bytes(HD);
    const float* sc = reinterpret_cast<const float*>(blk + 2 * kPage * HD);
    for (int t = 0; t < kPage; ++t) {
      const int pos = lp * kPage + t;
      if (pos > p || pos >= n || (a.window > 0 && pos <= p - a.window)) continue;
      float x = 0.f;
      #pragma unroll
      for (int d = 0; d < DPL; ++d) {
        const int dd = lane * DPL + d;
        const uint32_t w = *reinterpret_cast<const uint32_t*>(blk + kv8_k_at(t, dd & ~3));
        const float4 y = kv8_decode4<TYPE>(w);
        const float kk = (dd & 3) == 0 ? y.x : (dd & 3) == 1 ? y.y : (dd & 3) == 2 ? y.z : y.w;
        x = fmaf(qv[d], kk, x);
      }
      #pragma unroll
      for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
      x *= sc[0] * a.scale;
      if (a.cap > 0.f) x = a.cap * tanhf(x / a.cap);
      x = (x - slope * (float)(p - pos)) * 1.4426950408889634f;
      const float m_new = fmaxf(m, x), base = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m - base), w = exp2f(x - base);
      l = l * alpha + w;
      m = m_new;
      #pragma unroll
      for (int d = 0; d < DPL; ++d) {
        const int dd = lane * DPL + d;
        const uint32_t v = blk[kPage * HD + (dd >> 2) * 64 + (t >> 2) * 16 + (dd & 3) * 4 + (t & 3)];
        o[d] = o[d] * alpha + w * sc[1] * kv8_decode4<TYPE>(v).x;
      }
    }
  }
  #pragma unroll
  for (int d = 0; d < DPL; ++d) s_o[warp][lane * DPL + d] = o[d];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  T* out = static_cast<T*>(a.out) + (row * a.n_kv_heads * a.group + j) * HD;
  for (int d = threadIdx.x; d < HD; d += kKv8AttnWarps * 32) {
    float M = -INFINITY, L = 0.f, acc = 0.f;
    for (int w = 0; w < kKv8AttnWarps; ++w) M = fmaxf(M, s_m[w]);
    const float base = M == -INFINITY ? 0.f : M;
    for (int w = 0; w < kKv8AttnWarps; ++w) {
      const float f = exp2f(s_m[w] - base);
      L += f * s_l[w];
      acc += f * s_o[w][d];
    }
    const float y = L == 0.f ? 0.f : acc / L;
    out[d] = (T)y;
  }
}

}  // namespace bc

using namespace bc;

static bool attn8_sizes_ok(int batch, int H, int group, int max_q, int hd) {
  return batch >= 1 && batch <= BC_RAGGED_MAX_BATCH && H >= 1 && H <= 65535 && group >= 1 && group <= 8 && max_q >= 1 &&
         max_q <= 64 && group * max_q <= 64 && (hd == 64 || hd == 128);
}

extern "C" size_t bc_kv8_attention_scratch_bytes(int batch, int n_kv_heads, int group, int max_q, int head_dim) {
  if (!attn8_sizes_ok(batch, n_kv_heads, group, max_q, head_dim)) return 0;
  return 256;
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
  if (a->n_pages < 1 || a->n_pages > INT32_MAX / kPage || a->max_blocks < 1 || a->max_blocks > INT32_MAX / kPage ||
      a->n_q < 0 || (a->pages && a->max_sel < 1))
    return entry_fail(BC_EINVAL, "%s: bad page or row counts", who);
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
  const dim3 grid(a->n_kv_heads * a->group, a->batch * a->max_q), block(kKv8AttnWarps * 32);
  if ((long long)a->batch * a->max_q > 65535) return entry_fail(BC_EINVAL, "%s: batch * max_q above 65535", who);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
#define ATTN8(HD)                                                                                   \
  (a->type == BC_KV8_E4M3                                                                           \
       ? (a->dtype == BC_F32 ? launch_op(k_kv8_attn<HD, 0, float>, grid, block, 0, st, *a)          \
                             : launch_op(k_kv8_attn<HD, 0, __nv_bfloat16>, grid, block, 0, st, *a)) \
       : (a->dtype == BC_F32 ? launch_op(k_kv8_attn<HD, 1, float>, grid, block, 0, st, *a)          \
                             : launch_op(k_kv8_attn<HD, 1, __nv_bfloat16>, grid, block, 0, st, *a)))
  e = a->head_dim == 128 ? ATTN8(128) : ATTN8(64);
#undef ATTN8
  return entry_cuda(e, who);
}

extern "C" bc_status bc_kv8_attention_status(void* scratch, void* stream) {
  if (!scratch) return entry_fail(BC_EINVAL, "bc_kv8_attention_status: null scratch");
  return entry_cuda(cudaStreamSynchronize(static_cast<cudaStream_t>(stream)), "bc_kv8_attention_status");
}
