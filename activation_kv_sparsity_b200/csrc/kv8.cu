// Append to and read-back from the 8-bit paged cache.
//
// A block (page, kv head) has one scale for its 16 tokens' keys and one for
// their values:  code = rn(x * (1/s)),  s = max(s_old, m/Q),  m = max |x|.
// The work item of both kernels is one run of tokens with consecutive slots
// of one page, for one kv head, keys or values: a warp holds all of it in
// registers (lane: 4 dims of every token at head_dim 128; 4 dims of 8 tokens
// at 64), so m is one warp reduction and nothing is read twice.  Value codes
// lie four tokens to a word; the lane's 4 tokens x 4 dims are turned by byte
// permutes, and the lane's words are contiguous (16 bytes a group of tokens).
#include "entry.h"
#include "kv8.cuh"

namespace bc {

struct Kv8AppendArgs {
  const void *k, *v;
  long long k_stride, v_stride;
  const int* slots;
  int n_tokens, n_pages, H;
  uint8_t* pool;
  int window;     // tokens whose runs one warp handles
};

struct Kv8GatherArgs {
  const uint8_t* pool;
  int n_pages, H;
  const int* slots;
  int n_tokens;
  void *k, *v;
  int window;
};

constexpr int kKv8Threads = 128;

// The runs that begin in tokens [t0, t0 + window), window <= 16: calls
// body(first token, slot of it, tokens) for each, warp-uniform.  A run ends
// with its page.
template <typename F>
__device__ __forceinline__ void for_each_run(const int* slots, int n, int t0, int window, int n_slots, F body) {
  const int lane = threadIdx.x & 31;
  const int i = t0 - 1 + lane;                      // lane 0: the token before the window
  int s = i >= 0 && i < n ? slots[i] : -1;
  if (s >= n_slots) s = -1;
  const int prev = __shfl_up_sync(0xffffffffu, s, 1);
  const bool joins = lane > 0 && s >= 0 && prev >= 0 && s == prev + 1 && s % kPage != 0;
  const unsigned jm = __ballot_sync(0xffffffffu, joins);
  unsigned heads = __ballot_sync(0xffffffffu, s >= 0 && !joins && lane >= 1 && lane <= window);
  while (heads) {
    const int l = __ffs(heads) - 1;
    heads &= heads - 1;
    // lanes l + 1, l + 2, ... that join: at most 15, since a run ends with its page
    const unsigned follow = l < 31 ? ~(jm >> (l + 1)) : 1u;
    const int cnt = 1 + min(__ffs(follow) - 1, 31 - l);
    body(t0 - 1 + l, __shfl_sync(0xffffffffu, s, l), cnt);
  }
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

template <int HD, int TYPE, typename T>
__global__ void __launch_bounds__(kKv8Threads) k_kv8_append(Kv8AppendArgs a) {
  using C = Kv8Code<TYPE>;
  constexpr int LPT = HD / 4;          // lanes per token
  constexpr int NTOK = kPage * LPT / 32;   // tokens per lane
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kKv8Threads / 32) + (threadIdx.x >> 5);
  const int part = (int)(item & 1), h = (int)((item >> 1) % a.H);
  const long long t0 = (item >> 1) / a.H * a.window;
  pdl_wait();
  pdl_trigger();
  if (t0 >= a.n_tokens) return;
  const int d = (lane % LPT) * 4, p0 = (lane / LPT) * NTOK;
  const T* src = static_cast<const T*>(part ? a.v : a.k) + (long long)h * HD + d;
  const long long stride = part ? a.v_stride : a.k_stride;

  for_each_run(a.slots, a.n_tokens, (int)t0, a.window, a.n_pages * kPage, [&](int t, int slot, int cnt) {
    const int off = slot % kPage, end = off + cnt;
    uint8_t* blk = a.pool + ((long long)(slot / kPage) * a.H + h) * kv8_block_bytes(HD);
    float* scale = reinterpret_cast<float*>(blk + 2 * kPage * HD) + part;
    const float s_old = off > 0 ? *scale : 0.f;
    float4 x[NTOK];
    uint32_t top = 0;                  // |x| as an ordered integer: infinities and NaN come out on top
    #pragma unroll
    for (int i = 0; i < NTOK; ++i) {
      const int p = p0 + i;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p >= off && p < end) x[i] = load4<T>(src + (long long)(t + p - off) * stride);
      const uint32_t m = max(max(__float_as_uint(x[i].x) & 0x7fffffffu, __float_as_uint(x[i].y) & 0x7fffffffu),
                             max(__float_as_uint(x[i].z) & 0x7fffffffu, __float_as_uint(x[i].w) & 0x7fffffffu));
      top = max(top, m);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    float s;
    if (top >= 0x7f800000u || s_old != s_old) {
      s = __uint_as_float(0x7fc00000u);
    } else {
      s = top ? fmaxf(__fdiv_rn(__uint_as_float(top), C::kMax), 1.17549435e-38f) : 0.f;
      s = fmaxf(s_old, s);
    }
    const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
    const bool grown = off > 0 && s > s_old;
    uint32_t code[NTOK];
    #pragma unroll
    for (int i = 0; i < NTOK; ++i)
      code[i] = C::encode(x[i].x * inv, x[i].y * inv, x[i].z * inv, x[i].w * inv);
    auto again = [&](uint32_t w) {     // an earlier token's codes under the new scale
      const float4 y = kv8_decode4<TYPE>(w);
      return C::encode(y.x * s_old * inv, y.y * s_old * inv, y.z * s_old * inv, y.w * s_old * inv);
    };
    if (part == 0) {
      #pragma unroll
      for (int i = 0; i < NTOK; ++i) {
        const int p = p0 + i;
        uint32_t* dst = reinterpret_cast<uint32_t*>(blk + kv8_k_at(p, d));
        if (p < off) {
          if (grown) *dst = again(*dst);
        } else if (p < end || off == 0) {
          *dst = code[i];              // zeros behind the run of a fresh page
        }
      }
    } else {
      uint8_t* vb = blk + kPage * HD + d * kPage;
      #pragma unroll
      for (int g = 0; g < NTOK / 4; ++g) {
        const int p = p0 + 4 * g;
        uint4* dst = reinterpret_cast<uint4*>(vb + p * 4);
        const bool any = off == 0 || (p < end && (grown || p + 4 > off));
        if (!any) continue;
        uint32_t w[4] = {code[4 * g], code[4 * g + 1], code[4 * g + 2], code[4 * g + 3]};
        if (off > 0) {
          uint4 o4 = *dst;
          transpose4x4(o4.x, o4.y, o4.z, o4.w);
          const uint32_t old[4] = {o4.x, o4.y, o4.z, o4.w};
          #pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (p + j < off) w[j] = grown ? again(old[j]) : old[j];
            else if (p + j >= end) w[j] = old[j];
          }
        }
        transpose4x4(w[0], w[1], w[2], w[3]);
        *dst = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
    if (lane == 0) *scale = s;
  });
}

template <int HD, int TYPE, typename T>
__global__ void __launch_bounds__(kKv8Threads) k_kv8_gather(Kv8GatherArgs a) {
  constexpr int LPT = HD / 4;
  constexpr int NTOK = kPage * LPT / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * (kKv8Threads / 32) + (threadIdx.x >> 5);
  const int part = (int)(item & 1), h = (int)((item >> 1) % a.H);
  const long long t0 = (item >> 1) / a.H * a.window;
  pdl_wait();
  pdl_trigger();
  if (t0 >= a.n_tokens) return;
  const int d = (lane % LPT) * 4, p0 = (lane / LPT) * NTOK;
  T* out = static_cast<T*>(part ? a.v : a.k) + (long long)h * HD + d;
  const long long row = (long long)a.H * HD;
  // slots outside the pool give zeros
  for (int i = lane / LPT; i < a.window && t0 + i < a.n_tokens; i += 32 / LPT) {
    const int s = a.slots[t0 + i];
    if (s < 0 || s >= a.n_pages * kPage) store4(out + (t0 + i) * row, make_float4(0.f, 0.f, 0.f, 0.f));
  }
  for_each_run(a.slots, a.n_tokens, (int)t0, a.window, a.n_pages * kPage, [&](int t, int slot, int cnt) {
    const int off = slot % kPage, end = off + cnt;
    const uint8_t* blk = a.pool + ((long long)(slot / kPage) * a.H + h) * kv8_block_bytes(HD);
    const float s = reinterpret_cast<const float*>(blk + 2 * kPage * HD)[part];
    uint32_t w[NTOK];
    if (part == 0) {
      #pragma unroll
      for (int i = 0; i < NTOK; ++i) {
        const int p = p0 + i;
        w[i] = p >= off && p < end ? *reinterpret_cast<const uint32_t*>(blk + kv8_k_at(p, d)) : 0u;
      }
    } else {
      #pragma unroll
      for (int g = 0; g < NTOK / 4; ++g) {
        const int p = p0 + 4 * g;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (p < end && p + 4 > off) x = *reinterpret_cast<const uint4*>(blk + kPage * HD + d * kPage + p * 4);
        transpose4x4(x.x, x.y, x.z, x.w);
        w[4 * g] = x.x;
        w[4 * g + 1] = x.y;
        w[4 * g + 2] = x.z;
        w[4 * g + 3] = x.w;
      }
    }
    #pragma unroll
    for (int i = 0; i < NTOK; ++i) {
      const int p = p0 + i;
      if (p >= off && p < end) {
        const float4 y = kv8_decode4<TYPE>(w[i]);
        store4(out + (long long)(t + p - off) * row, make_float4(y.x * s, y.y * s, y.z * s, y.w * s));
      }
    }
  });
}

}  // namespace bc

using namespace bc;

static bool kv8_sizes_ok(int n_pages, int H, int hd) {
  return n_pages >= 1 && n_pages <= INT32_MAX / kPage && H >= 1 && H <= 65535 && (hd == 64 || hd == 128);
}

static bc_status kv8_check(const char* who, const void* pool, int type, int n_pages, int H, int hd, int dtype,
                           int n_tokens) {
  if (!pool) return entry_fail(BC_EINVAL, "%s: null pool", who);
  if (!aligned(pool, 16)) return entry_fail(BC_EINVAL, "%s: the pool must be 16-byte aligned", who);
  if (hd != 64 && hd != 128) return entry_fail(BC_EINVAL, "%s: head_dim must be 64 or 128", who);
  if (!kv8_sizes_ok(n_pages, H, hd)) return entry_fail(BC_EINVAL, "%s: bad n_pages or n_kv_heads", who);
  if (type != BC_KV8_E4M3 && type != BC_KV8_INT8) return entry_fail(BC_EINVAL, "%s: bad code type %d", who, type);
  if (dtype != BC_F32 && dtype != BC_BF16) return entry_fail(BC_EINVAL, "%s: bad dtype %d", who, dtype);
  if (n_tokens < 0) return entry_fail(BC_EINVAL, "%s: n_tokens < 0", who);
  return BC_OK;
}

// One token a warp while that leaves the GPU room, else a page's worth of
// tokens (whose runs, one or two for a prompt, the warp takes in turn).
static int kv8_window(int n_tokens) { return n_tokens <= 2048 ? 1 : kPage; }

static bc_status kv8_grid(const char* who, int n_tokens, int window, int H, unsigned* grid) {
  const long long warps = (n_tokens + (long long)window - 1) / window * H * 2;
  const long long g = (warps + kKv8Threads / 32 - 1) / (kKv8Threads / 32);
  if (g > INT32_MAX) return entry_fail(BC_EINVAL, "%s: too many tokens and heads for one call", who);
  *grid = (unsigned)g;
  return BC_OK;
}

#define KV8_LAUNCH(KERN, ...)                                                                                \
  do {                                                                                                       \
    if (head_dim == 128) {                                                                                   \
      if (type == BC_KV8_E4M3)                                                                               \
        e = dtype == BC_F32 ? launch_op(KERN<128, 0, float>, __VA_ARGS__)                                    \
                            : launch_op(KERN<128, 0, __nv_bfloat16>, __VA_ARGS__);                           \
      else                                                                                                   \
        e = dtype == BC_F32 ? launch_op(KERN<128, 1, float>, __VA_ARGS__)                                    \
                            : launch_op(KERN<128, 1, __nv_bfloat16>, __VA_ARGS__);                           \
    } else {                                                                                                 \
      if (type == BC_KV8_E4M3)                                                                               \
        e = dtype == BC_F32 ? launch_op(KERN<64, 0, float>, __VA_ARGS__)                                     \
                            : launch_op(KERN<64, 0, __nv_bfloat16>, __VA_ARGS__);                            \
      else                                                                                                   \
        e = dtype == BC_F32 ? launch_op(KERN<64, 1, float>, __VA_ARGS__)                                     \
                            : launch_op(KERN<64, 1, __nv_bfloat16>, __VA_ARGS__);                            \
    }                                                                                                        \
  } while (0)

extern "C" size_t bc_kv8_pool_bytes(int n_pages, int n_kv_heads, int head_dim) {
  if (!kv8_sizes_ok(n_pages, n_kv_heads, head_dim)) return 0;
  return (size_t)n_pages * n_kv_heads * kv8_block_bytes(head_dim);
}

extern "C" bc_status bc_kv8_append(const void* k, const void* v, bc_dtype dtype, long long k_stride,
                                   long long v_stride, const int* slots, int n_tokens, void* pool, bc_kv8_type type,
                                   int n_pages, int n_kv_heads, int head_dim, void* stream) {
  const char* who = "bc_kv8_append";
  bc_status s = kv8_check(who, pool, type, n_pages, n_kv_heads, head_dim, dtype, n_tokens);
  if (s != BC_OK) return s;
  if (n_tokens == 0) return BC_OK;
  if (!k || !v || !slots) return entry_fail(BC_EINVAL, "%s: null pointer", who);
  const size_t al = dtype == BC_F32 ? 16 : 8;
  if (!aligned(k, al) || !aligned(v, al)) return entry_fail(BC_EINVAL, "%s: k and v must be %zu-byte aligned", who, al);
  const long long least = (long long)n_kv_heads * head_dim;
  if (k_stride < least || v_stride < least || k_stride % 4 || v_stride % 4)
    return entry_fail(BC_EINVAL, "%s: strides must be multiples of 4 and at least n_kv_heads * head_dim", who);
  Kv8AppendArgs a{k, v, k_stride, v_stride, slots, n_tokens, n_pages, n_kv_heads, static_cast<uint8_t*>(pool),
                  kv8_window(n_tokens)};
  unsigned grid;
  s = kv8_grid(who, n_tokens, a.window, n_kv_heads, &grid);
  if (s != BC_OK) return s;
  cudaError_t e;
  KV8_LAUNCH(k_kv8_append, dim3(grid), dim3(kKv8Threads), 0, static_cast<cudaStream_t>(stream), a);
  return entry_cuda(e, who);
}

extern "C" bc_status bc_kv8_gather(const void* pool, bc_kv8_type type, int n_pages, int n_kv_heads, int head_dim,
                                   const int* slots, int n_tokens, void* k_out, void* v_out, bc_dtype dtype,
                                   void* stream) {
  const char* who = "bc_kv8_gather";
  bc_status s = kv8_check(who, pool, type, n_pages, n_kv_heads, head_dim, dtype, n_tokens);
  if (s != BC_OK) return s;
  if (n_tokens == 0) return BC_OK;
  if (!k_out || !v_out || !slots) return entry_fail(BC_EINVAL, "%s: null pointer", who);
  if (!aligned(k_out, 16) || !aligned(v_out, 16))
    return entry_fail(BC_EINVAL, "%s: outputs must be 16-byte aligned", who);
  Kv8GatherArgs a{static_cast<const uint8_t*>(pool), n_pages, n_kv_heads, slots, n_tokens, k_out, v_out,
                  kv8_window(n_tokens)};
  unsigned grid;
  s = kv8_grid(who, n_tokens, a.window, n_kv_heads, &grid);
  if (s != BC_OK) return s;
  cudaError_t e;
  KV8_LAUNCH(k_kv8_gather, dim3(grid), dim3(kKv8Threads), 0, static_cast<cudaStream_t>(stream), a);
  return entry_cuda(e, who);
}
