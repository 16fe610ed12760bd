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
// HBM bounds both for prompts, the chain slots - tokens - scale - codes a
// decode step.  A CTA takes a window of tokens and a group of heads; its
// warps share the items of the runs that begin there.  Graph replays, 8 heads of
// 128: 32768 tokens read back as bf16 in 36 us (5.6 TB/s), 23 thousand appended
// from bf16 in 29 us (4.9 TB/s), from f32 in 41 us (5.7 TB/s); 256 tokens to as
// many pages 6.6 us.  80 registers a thread, for three CTAs an SM, spill a few
// words: 60 bytes in the append of f32 at head_dim 128, 4 to 20 in its other
// forms and in the read-back there, none at 64.  Persistent CTAs spilled more and
// were slower.
#include "entry.h"
#include "kv8.cuh"

#include <algorithm>
#include <type_traits>

namespace bc {

struct Kv8AppendArgs {
  const void *k, *v;
  long long k_stride, v_stride;
  const int* slots;
  int n_tokens, n_pages, H;
  uint8_t* pool;
  int window, heads;     // tokens and kv heads per CTA
};

struct Kv8GatherArgs {
  const uint8_t* pool;
  int n_pages, H;
  const int* slots;
  int n_tokens;
  void *k, *v;
  int window, heads;
};

constexpr int kKv8Warps = 8, kKv8Threads = kKv8Warps * 32, kKv8Ctas = 3;   // CTAs per SM

// The runs that begin in tokens [t0, t0 + window), window <= 16, and for each
// the 2 * heads items of keys and values: calls body(first token, slot of it,
// tokens, item) for this warp's share.  A run ends with its page.
template <typename F>
__device__ __forceinline__ void for_each_item(const int* slots, int n, int t0, int window, int n_slots, int items,
                                              F body) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = t0 - 1 + lane;                      // lane 0: the token before the window
  int s = i >= 0 && i < n ? slots[i] : -1;
  if (s >= n_slots) s = -1;
  const int prev = __shfl_up_sync(0xffffffffu, s, 1);
  const bool joins = lane > 0 && s >= 0 && prev >= 0 && s == prev + 1 && s % kPage != 0;
  const unsigned jm = __ballot_sync(0xffffffffu, joins);
  unsigned heads = __ballot_sync(0xffffffffu, s >= 0 && !joins && lane >= 1 && lane <= window);
  int item = warp;                                  // of all runs' items, one after the other
  while (heads) {
    const int l = __ffs(heads) - 1;
    heads &= heads - 1;
    // lanes l + 1, l + 2, ... that join: at most 15, since a run ends with its page
    const unsigned follow = l < 31 ? ~(jm >> (l + 1)) : 1u;
    const int cnt = 1 + min(__ffs(follow) - 1, 31 - l), slot = __shfl_sync(0xffffffffu, s, l);
    for (; item < items; item += kKv8Warps) body(t0 - 1 + l, slot, cnt, item);
    item -= items;
  }
}

// Four neighbouring elements as loaded: their values, and the largest |x| as
// an ordered integer (infinities and NaN come out on top).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  uint4 w;
  __device__ __forceinline__ void load(const float* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ __forceinline__ void top(uint32_t& t) const {
    t = max(t, max(max(w.x & 0x7fffffffu, w.y & 0x7fffffffu), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu)));
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t t) { return t; }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint2(0, 0); }
  __device__ __forceinline__ float4 get() const { return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)); }
  // two 16-bit maxima side by side
  __device__ __forceinline__ void top(uint32_t& t) const {
    t = __vmaxu2(t, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t t) { return max(t & 0xffffu, t >> 16) << 16; }
};
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
}

template <int HD, int TYPE, typename T>
__global__ void __launch_bounds__(kKv8Threads, kKv8Ctas) k_kv8_append(Kv8AppendArgs a) {
  using C = Kv8Code<TYPE>;
  constexpr int LPT = HD / 4;          // lanes per token
  constexpr int NTOK = kPage * LPT / 32;   // tokens per lane
  const int lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.window, head0 = blockIdx.y * a.heads;
  pdl_wait();
  pdl_trigger();
  const int d = (lane % LPT) * 4, p0 = (lane / LPT) * NTOK;

  for_each_item(a.slots, a.n_tokens, t0, a.window, a.n_pages * kPage, 2 * min(a.heads, a.H - head0),
                [&](int t, int slot, int cnt, int item) {
    const int part = item & 1, h = head0 + (item >> 1), off = slot % kPage, end = off + cnt;
    const long long stride = part ? a.v_stride : a.k_stride;
    // the lane's first token, if it were one of the run
    const T* src = static_cast<const T*>(part ? a.v : a.k) + (long long)h * HD + d + (t + p0 - off) * stride;
    uint8_t* blk = a.pool + ((long long)(slot / kPage) * a.H + h) * kv8_block_bytes(HD);
    float* scale = reinterpret_cast<float*>(blk + 2 * kPage * HD) + part;
    // a whole page (most of a prompt) needs no questions about its tokens
    auto write = [&](auto whole_page) {
      constexpr bool WHOLE = decltype(whole_page)::value;
      const float s_old = !WHOLE && off > 0 ? *scale : 0.f;
      Raw<T> raw[NTOK];
      uint32_t top = 0;
      #pragma unroll
      for (int i = 0; i < NTOK; ++i) {
        raw[i].zero();
        if (WHOLE || (p0 + i >= off && p0 + i < end)) raw[i].load(src + i * stride);
      }
      #pragma unroll
      for (int i = 0; i < NTOK; ++i) raw[i].top(top);
      top = __reduce_max_sync(0xffffffffu, Raw<T>::bits(top));
      float s;
      if (top >= 0x7f800000u || s_old != s_old) {
        s = __uint_as_float(0x7fc00000u);
      } else {
        s = top ? fmaxf(__fdiv_rn(__uint_as_float(top), C::kMax), 1.17549435e-38f) : 0.f;
        s = fmaxf(s_old, s);
      }
      const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
      const bool grown = !WHOLE && off > 0 && s > s_old;
      uint32_t code[NTOK];
      #pragma unroll
      for (int i = 0; i < NTOK; ++i) {
        const float4 x = raw[i].get();
        // zeros under a scale that is not a number, whatever x is: a code that
        // is none would reach rows that mask the token
        const uint32_t c = C::encode(__fmul_rn(x.x, inv), __fmul_rn(x.y, inv), __fmul_rn(x.z, inv), __fmul_rn(x.w, inv));
        code[i] = inv > 0.f ? c : 0u;
      }
      auto again = [&](uint32_t w) {     // an earlier token's codes under the new scale
        const float4 y = kv8_decode4<TYPE>(w);
        auto f = [&](float v) { return __fmul_rn(__fmul_rn(v, s_old), inv); };
        return C::encode(f(y.x), f(y.y), f(y.z), f(y.w));
      };
      if (part == 0) {
        uint8_t* kb = blk + kv8_k_at(p0, d);
        #pragma unroll
        for (int i = 0; i < NTOK; ++i) {
          uint32_t* dst = reinterpret_cast<uint32_t*>(kb + 64 * i);
          if (!WHOLE && p0 + i < off) {
            if (grown) *dst = again(*dst);
          } else if (WHOLE || p0 + i < end || off == 0) {
            *dst = code[i];              // zeros behind the run of a fresh page
          }
        }
      } else {
        uint8_t* vb = blk + kPage * HD + d * kPage + p0 * 4;
        #pragma unroll
        for (int g = 0; g < NTOK / 4; ++g) {
          const int p = p0 + 4 * g;
          uint4* dst = reinterpret_cast<uint4*>(vb + 16 * g);
          if (!WHOLE && off > 0 && (p >= end || (!grown && p + 4 <= off))) continue;
          uint32_t w[4] = {code[4 * g], code[4 * g + 1], code[4 * g + 2], code[4 * g + 3]};
          if (!WHOLE && off > 0) {
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
    };
    if (cnt == kPage) write(std::true_type{});
    else write(std::false_type{});
  });
}

template <int HD, int TYPE, typename T>
__global__ void __launch_bounds__(kKv8Threads, kKv8Ctas) k_kv8_gather(Kv8GatherArgs a) {
  constexpr int LPT = HD / 4;
  constexpr int NTOK = kPage * LPT / 32;
  const int lane = threadIdx.x & 31;
  const int t0 = blockIdx.x * a.window, head0 = blockIdx.y * a.heads, heads = min(a.heads, a.H - head0);
  pdl_wait();
  pdl_trigger();
  const int d = (lane % LPT) * 4, p0 = (lane / LPT) * NTOK;
  const long long row = (long long)a.H * HD;
  // slots outside the pool give zeros
  for (int i = threadIdx.x >> 5; i < a.window && t0 + i < a.n_tokens; i += kKv8Warps) {
    const int s = a.slots[t0 + i];
    if (s >= 0 && s < a.n_pages * kPage) continue;
    for (int e = 4 * lane; e < heads * HD; e += 128) {
      store4(static_cast<T*>(a.k) + (t0 + i) * row + head0 * HD + e, make_float4(0.f, 0.f, 0.f, 0.f));
      store4(static_cast<T*>(a.v) + (t0 + i) * row + head0 * HD + e, make_float4(0.f, 0.f, 0.f, 0.f));
    }
  }
  for_each_item(a.slots, a.n_tokens, t0, a.window, a.n_pages * kPage, 2 * heads,
                [&](int t, int slot, int cnt, int item) {
    const int part = item & 1, h = head0 + (item >> 1), off = slot % kPage, end = off + cnt;
    const uint8_t* blk = a.pool + ((long long)(slot / kPage) * a.H + h) * kv8_block_bytes(HD);
    // the lane's first token, if it were one of the run
    T* out = static_cast<T*>(part ? a.v : a.k) + (long long)h * HD + d + (t + p0 - off) * row;
    auto read = [&](auto whole_page) {
      constexpr bool WHOLE = decltype(whole_page)::value;
      const float s = reinterpret_cast<const float*>(blk + 2 * kPage * HD)[part];
      uint32_t w[NTOK];
      if (part == 0) {
        const uint8_t* kb = blk + kv8_k_at(p0, d);
        #pragma unroll
        for (int i = 0; i < NTOK; ++i)
          w[i] = WHOLE || (p0 + i >= off && p0 + i < end) ? *reinterpret_cast<const uint32_t*>(kb + 64 * i) : 0u;
      } else {
        const uint8_t* vb = blk + kPage * HD + d * kPage + p0 * 4;
        uint4 x[NTOK / 4];
        #pragma unroll
        for (int g = 0; g < NTOK / 4; ++g) {
          x[g] = make_uint4(0, 0, 0, 0);
          if (WHOLE || (p0 + 4 * g < end && p0 + 4 * g + 4 > off)) x[g] = *reinterpret_cast<const uint4*>(vb + 16 * g);
        }
        #pragma unroll
        for (int g = 0; g < NTOK / 4; ++g) {
          transpose4x4(x[g].x, x[g].y, x[g].z, x[g].w);
          w[4 * g] = x[g].x;
          w[4 * g + 1] = x[g].y;
          w[4 * g + 2] = x[g].z;
          w[4 * g + 3] = x[g].w;
        }
      }
      #pragma unroll
      for (int i = 0; i < NTOK; ++i) {
        if (!WHOLE && (p0 + i < off || p0 + i >= end)) continue;
        const float4 y = kv8_decode4<TYPE>(w[i]);
        store4(out + i * row, make_float4(y.x * s, y.y * s, y.z * s, y.w * s));
      }
    };
    if (cnt == kPage) read(std::true_type{});
    else read(std::false_type{});
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
  if (n_tokens < 0 || n_tokens > INT32_MAX - 64) return entry_fail(BC_EINVAL, "%s: bad n_tokens %d", who, n_tokens);
  return BC_OK;
}

// Windows of a page's worth of tokens (one or two runs of a prompt) and 8
// heads, of fewer heads and then of 4 tokens (a decode step has a run a token)
// until there is a CTA for every place on the GPU.
static dim3 kv8_grid(int n_tokens, int H, int* window, int* heads) {
  constexpr long long kPlaces = 148 * kKv8Ctas;
  *window = kPage;
  *heads = std::min(H, 8);
  auto windows = [&]() { return (n_tokens + (long long)*window - 1) / *window; };
  auto groups = [&]() { return (H + *heads - 1) / *heads; };
  while (*heads > 1 && windows() * groups() < kPlaces) *heads = (*heads + 1) / 2;
  while (*window > 4 && windows() * groups() < kPlaces) *window /= 2;
  return dim3((unsigned)windows(), (unsigned)groups());
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
  Kv8AppendArgs a{k, v, k_stride, v_stride, slots, n_tokens, n_pages, n_kv_heads, static_cast<uint8_t*>(pool), 0, 0};
  const dim3 grid = kv8_grid(n_tokens, n_kv_heads, &a.window, &a.heads);
  cudaError_t e;
  KV8_LAUNCH(k_kv8_append, grid, dim3(kKv8Threads), 0, static_cast<cudaStream_t>(stream), a);
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
  Kv8GatherArgs a{static_cast<const uint8_t*>(pool), n_pages, n_kv_heads, slots, n_tokens, k_out, v_out, 0, 0};
  const dim3 grid = kv8_grid(n_tokens, n_kv_heads, &a.window, &a.heads);
  cudaError_t e;
  KV8_LAUNCH(k_kv8_gather, grid, dim3(kKv8Threads), 0, static_cast<cudaStream_t>(stream), a);
  return entry_cuda(e, who);
}
