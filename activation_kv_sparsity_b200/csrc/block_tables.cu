// The plan of one step of a ragged batch (bc_block_tables): which pages each
// sequence gives back or takes, and where each new token goes.
//
// With h_b = ceil(n_b / 16) pages held, the plan is three running sums over
// the sequences, of the new tokens asked for, of the pages needed and given
// back, and of the tokens granted and the pages taken.  Every CTA computes
// all three by itself (2048 sequences are 8 KB to read, against a second
// kernel or a grid-wide wait), keeps them in shared memory, and writes its
// share of the tokens, table entries and free pages; each of those finds its
// sequence by a binary search of the sums.  Reads and writes of the tables
// never meet: old entries are read, new ones written, and the page of a new
// token is taken from the free list, not from the table.  Only lens_out and
// n_free_out may lie on inputs; the last CTA to finish (an atomic ticket, no
// spinning) writes them.  Graph replays: 4.2 us for 24 requests that take a token
// each, the latency of a launch and three sums; 10.9 us for 1000 that take 190
// thousand, 3.9 million warp instructions (half the issue slots), most of them the
// ten steps of a search for every token and the sums, which every CTA repeats.
#include "common.cuh"
#include "entry.h"

#include <algorithm>

namespace bc {

// Threads of a CTA: the sums of a small batch take few warps.
constexpr int kPlanSmall = 128, kPlanLarge = 1024;
constexpr int kPlanTokens = 2;     // tokens per thread in flight

struct Sum2 {
  long long a, b;
};

// Exclusive running sums of a pair over the block; *total receives the sums.
template <int NT>
__device__ __forceinline__ Sum2 block_scan2(Sum2 v, Sum2* red, Sum2* total) {
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  Sum2 x = v;
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, x.a, o), b = __shfl_up_sync(0xffffffffu, x.b, o);
    if (l >= o) {
      x.a += a;
      x.b += b;
    }
  }
  if (l == 31) red[w] = x;
  __syncthreads();
  if (w == 0) {
    Sum2 t = l < NT / 32 ? red[l] : Sum2{0, 0};
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, t.a, o), b = __shfl_up_sync(0xffffffffu, t.b, o);
      if (l >= o) {
        t.a += a;
        t.b += b;
      }
    }
    red[l] = t;
  }
  __syncthreads();
  Sum2 before = {0, 0};
  if (w > 0) before = red[w - 1];
  *total = red[NT / 32 - 1];
  __syncthreads();
  return Sum2{before.a + x.a - v.a, before.b + x.b - v.b};
}

// The last index b in [0, n) with sums[b] <= x (sums ascending, sums[0] <= x).
__device__ __forceinline__ int find_seq(const int* sums, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_of(long long n) { return (int)((n + kPage - 1) / kPage); }

template <int NT, int ITEMS>
__global__ void __launch_bounds__(NT) k_block_tables(const __grid_constant__ bc_block_tables_args a) {
  extern __shared__ int sm[];
  const int B = a.batch;
  int* s_len = sm;                 // [B] tokens held
  int* s_start = s_len + B;        // [B + 1] running sum of the tokens granted
  int* s_take = s_start + B + 1;   // [B + 1] of the pages taken
  int* s_back = s_take + B + 1;    // [B + 1] of the pages given back
  __shared__ Sum2 red[32];
  __shared__ int s_last;
  pdl_wait();
  pdl_trigger();

  const long long cap = (long long)a.max_blocks * kPage;
  const int n_free = min(max(*a.n_free, 0), a.n_pages);
  long long len[ITEMS], now[ITEMS], cand[ITEMS], need[ITEMS], back[ITEMS];
  Sum2 mine = {0, 0}, total;
  #pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int b = threadIdx.x * ITEMS + i;
    len[i] = now[i] = cand[i] = need[i] = back[i] = 0;
    if (b < B) {
      const long long d = a.delta[b];
      len[i] = min(max((long long)a.lens[b], 0LL), cap);
      now[i] = d < 0 ? max(len[i] + d, 0LL) : len[i];
      back[i] = pages_of(len[i]) - pages_of(now[i]);
      cand[i] = d > 0 && len[i] + d <= cap ? d : 0;
    }
    mine.a += cand[i];
    mine.b += back[i];
  }
  const Sum2 s1 = block_scan2<NT>(mine, red, &total);
  const long long n_back = total.b;
  // at most n_pages free pages (more would mean a page held twice)
  const int room = (int)min(n_free + n_back, (long long)a.n_pages);
  long long at = s1.a, rel = s1.b;
  mine.a = mine.b = 0;
  #pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int b = threadIdx.x * ITEMS + i;
    at += cand[i];
    if (at > a.max_tokens) cand[i] = 0;
    need[i] = cand[i] ? pages_of(len[i] + cand[i]) - pages_of(len[i]) : 0;
    mine.a += need[i];
    // (exact for the sequences that the list has room for: rooms and a
    // sequence's pages are at most 2^27)
    if (b < B) s_back[b] = (int)min(rel, (long long)INT32_MAX);
    rel += back[i];
  }
  const Sum2 s2 = block_scan2<NT>(mine, red, &total);
  at = s2.a;
  mine.a = mine.b = 0;
  #pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    at += need[i];
    if (need[i] && at > room) cand[i] = need[i] = 0;
    mine.a += cand[i];
    mine.b += need[i];
  }
  const Sum2 s3 = block_scan2<NT>(mine, red, &total);
  const int n_tok = (int)total.a, n_take = (int)total.b;
  long long tok = s3.a, take = s3.b;
  #pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int b = threadIdx.x * ITEMS + i;
    if (b < B) {
      s_len[b] = (int)len[i];
      s_start[b] = (int)tok;
      s_take[b] = (int)take;
      if (blockIdx.x == 0) a.q_start[b] = (int)tok;
      now[i] += cand[i];
    }
    tok += cand[i];
    take += need[i];
  }
  if (threadIdx.x == 0) {
    s_start[B] = n_tok;
    s_take[B] = n_take;
    s_back[B] = (int)min(n_back, (long long)INT32_MAX);
    if (blockIdx.x == 0) a.q_start[B] = n_tok;
  }
  __syncthreads();

  // page x of the free list followed by the pages given back
  auto free_page = [&](int x) {
    if (x < n_free) return a.free_list[x];
    const int r = x - n_free, b = find_seq(s_back, B, r);
    const int kept = pages_of(s_len[b]) - (s_back[b + 1] - s_back[b]);
    return a.table[(size_t)b * a.max_blocks + kept + (r - s_back[b])];
  };
  const int t0 = blockIdx.x * NT + threadIdx.x, step = gridDim.x * NT;
  for (long long i0 = t0; i0 < a.max_tokens; i0 += (long long)kPlanTokens * step) {
    int pos[kPlanTokens], page[kPlanTokens];
    #pragma unroll
    for (int j = 0; j < kPlanTokens; ++j) {
      const long long i = i0 + (long long)j * step;
      pos[j] = page[j] = -1;
      if (i < n_tok) {
        const int b = find_seq(s_start, B, (int)i);
        pos[j] = s_len[b] + (int)i - s_start[b];
        const int blk = pos[j] / kPage, held = pages_of(s_len[b]);
        page[j] = blk < held ? a.table[(size_t)b * a.max_blocks + blk] : free_page(room - 1 - (s_take[b] + blk - held));
      }
    }
    #pragma unroll
    for (int j = 0; j < kPlanTokens; ++j) {
      const long long i = i0 + (long long)j * step;
      if (i >= a.max_tokens) break;
      a.slots[i] = page[j] >= 0 && page[j] < a.n_pages ? page[j] * kPage + pos[j] % kPage : -1;
      a.positions[i] = pos[j];
    }
  }
  for (int j = t0; j < n_take; j += step) {
    const int b = find_seq(s_take, B, j);
    a.table[(size_t)b * a.max_blocks + pages_of(s_len[b]) + (j - s_take[b])] = free_page(room - 1 - j);
  }
  for (int x = n_free + t0; x < room - n_take; x += step) a.free_list[x] = free_page(x);

  // every CTA has read its inputs once the last one is here
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned prev;
    asm volatile("atom.add.acq_rel.gpu.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.ticket) : "memory");
    s_last = prev == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  #pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int b = threadIdx.x * ITEMS + i;
    if (b < B) a.lens_out[b] = (int)now[i];
  }
  if (threadIdx.x == 0) {
    *a.n_free_out = room - n_take;
    *a.ticket = 0u;
  }
}

}  // namespace bc

using namespace bc;

extern "C" bc_status bc_block_tables(const bc_block_tables_args* a, void* stream) {
  if (!a) return entry_fail(BC_EINVAL, "bc_block_tables: null arguments");
  if (!a->lens || !a->delta || !a->table || !a->free_list || !a->n_free || !a->lens_out || !a->n_free_out ||
      !a->q_start || !a->ticket || (a->max_tokens > 0 && (!a->slots || !a->positions)))
    return entry_fail(BC_EINVAL, "bc_block_tables: null pointer");
  if (a->batch < 1 || a->batch > BC_RAGGED_MAX_BATCH)
    return entry_fail(BC_EINVAL, "bc_block_tables: batch %d outside [1, %d]", a->batch, BC_RAGGED_MAX_BATCH);
  if (a->max_blocks < 1 || a->max_blocks > INT32_MAX / kPage)
    return entry_fail(BC_EINVAL, "bc_block_tables: bad max_blocks %d", a->max_blocks);
  if (a->n_pages < 1 || a->n_pages > INT32_MAX / kPage)
    return entry_fail(BC_EINVAL, "bc_block_tables: bad n_pages %d", a->n_pages);
  if (a->max_tokens < 0) return entry_fail(BC_EINVAL, "bc_block_tables: max_tokens < 0");
  const size_t smem = 4ull * (4 * (size_t)a->batch + 3);
  // kPlanTokens tokens a thread: the sums cost every CTA the same, so more
  // CTAs only shorten the token loop
  const int nt = a->batch <= kPlanSmall && a->max_tokens <= 4 * kPlanSmall ? kPlanSmall : kPlanLarge;
  const long long per = (long long)nt * kPlanTokens;
  const dim3 grid((unsigned)std::min(148LL, std::max(1LL, (a->max_tokens + per - 1) / per)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return entry_cuda(nt == kPlanSmall ? launch_op(k_block_tables<kPlanSmall, 1>, grid, dim3(nt), smem, st, *a)
                                     : launch_op(k_block_tables<kPlanLarge, BC_RAGGED_MAX_BATCH / kPlanLarge>, grid,
                                                 dim3(nt), smem, st, *a), "bc_block_tables");
}
