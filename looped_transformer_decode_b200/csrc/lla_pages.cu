// Pages of a cache shared by sequences of different lengths: block tables, the free
// list and the slot map of new tokens, kept on the GPU from how much each sequence
// grows or shrinks.
//
// Sequence b of length L holds its tokens in the pages block_table[b][0 .. ceil(L/P)).
// A call first takes back the pages of sequences that shrink, then serves the growing
// ones in order.  Everything is a prefix sum over the sequences:
//   need(b)  = ceil(new/P) - ceil(old/P)       pages
//   page k of b's need = free_list[n_free - 1 - (need before b) - k]
// and pages given back land where a growth of the same size would take them from, so
// that dropping the tokens just added restores the free list.
//
// pages_kernel (one block) does the sequences; the slots of the tokens, position by
// position, follow in it or, for many tokens, in pages_fill_kernel.
#include "lla_internal.cuh"

namespace lla {
namespace {

constexpr int kPagesThreads = 1024;

__device__ __forceinline__ int pages_of(long long len, int shift) {
  return (int)((len + (1 << shift) - 1) >> shift);
}

// Inclusive prefix sum of v over the block, and the block's total.
__device__ __forceinline__ long long block_scan(long long v, long long* warp_sums,
                                                long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < kPagesThreads / 32; ++w) {
    const long long t = warp_sums[w];
    if (w < warp) before += t;
    all += t;
  }
  __syncthreads();
  *total = all;
  return v + before;
}

// Slots and positions of tokens i, i + step, ... < tok_cap.
__device__ __forceinline__ void fill_tokens(const PageMapArgs& a, long long i0, long long step) {
  const int total = a.tok_start[a.B];
  const int P = 1 << a.shift;
  for (long long i = i0; i < a.tok_cap; i += step) {
    if (i >= total) {
      a.slot[i] = -1;
      a.positions[i] = 0;
      continue;
    }
    int lo = 0, hi = a.B;                       // tok_start[lo] <= i < tok_start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.tok_start[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int pos = a.ctx_len[lo] - (a.tok_start[lo + 1] - (int)i);
    const int page = a.block_table[(long long)lo * a.max_pages + (pos >> a.shift)];
    const bool known = page >= 0 && page < a.n_pages;
    if (!known && a.status) atomicOr(a.status, LLA_STATUS_PAGE_RANGE);
    a.slot[i] = known ? ((long long)page << a.shift) + (pos & (P - 1)) : -1;
    a.positions[i] = pos;
  }
}

__global__ void __launch_bounds__(kPagesThreads) pages_kernel(PageMapArgs a) {
  __shared__ long long warp_sums[kPagesThreads / 32];
  const int lane = threadIdx.x & 31;
  const long long limit = (long long)a.max_pages << a.shift;
  int nf = *a.n_free;
  int bits = 0;
  if (nf < 0 || nf > a.n_pages) {
    bits |= LLA_STATUS_PAGE_RANGE;
    nf = nf < 0 ? 0 : a.n_pages;
  }

  // old and new length of sequence b; a length outside its table is left alone
  auto lengths = [&](int b, long long& old_len, long long& new_len) {
    old_len = new_len = 0;
    if (b >= a.B) return;
    old_len = a.ctx_len[b];
    if (old_len < 0 || old_len > limit) {
      bits |= LLA_STATUS_CTX_RANGE;
      new_len = old_len;
      return;
    }
    new_len = old_len + a.n_new[b];
    if (new_len < 0) new_len = 0;
    if (new_len > limit) {
      bits |= LLA_STATUS_CTX_RANGE;
      new_len = old_len;
    }
  };

  // pages given back, counted first: they are pushed in reverse
  long long gone = 0, shrinking = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPagesThreads) {
    long long o, n, t;
    lengths(b0 + threadIdx.x, o, n);
    // pages below bit 40, sequences above it
    block_scan(n < o ? (1LL << 40) + pages_of(o, a.shift) - pages_of(n, a.shift) : 0, warp_sums, &t);
    gone += t & ((1LL << 40) - 1);
    shrinking += t >> 40;
  }
  if (shrinking) {
    long long carry = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPagesThreads) {
      const int b = b0 + threadIdx.x;
      long long o, n, t;
      lengths(b, o, n);
      const int first = pages_of(n, a.shift);
      const int back = n < o ? pages_of(o, a.shift) - first : 0;
      const long long at = carry + block_scan(back, warp_sums, &t) - back;
      carry += t;
      for (unsigned m = __ballot_sync(0xffffffffu, back > 0); m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const int bb = __shfl_sync(0xffffffffu, b, l), ff = __shfl_sync(0xffffffffu, first, l);
        const int cc = __shfl_sync(0xffffffffu, back, l);
        const long long aa = __shfl_sync(0xffffffffu, at, l);
        for (int k = lane; k < cc; k += 32) {
          int32_t* entry = a.block_table + (long long)bb * a.max_pages + ff + k;
          int page = *entry;
          *entry = -1;
          if (page < 0 || page >= a.n_pages) {
            bits |= LLA_STATUS_PAGE_RANGE;
            page = -1;
          }
          const long long to = nf + gone - 1 - (aa + k);
          if (to < a.n_pages) a.free_list[to] = page;
          else bits |= LLA_STATUS_PAGE_RANGE;
        }
      }
      if (n < o) a.ctx_len[b] = (int)n;
    }
    nf = (int)(nf + gone < a.n_pages ? nf + gone : a.n_pages);
  }
  __syncthreads();

  // growing sequences, in order: served while everything asked so far fits
  long long ask_pages = 0, ask_toks = 0, got_pages = 0, got_toks = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPagesThreads) {
    const int b = b0 + threadIdx.x;
    long long o, n, t;
    lengths(b, o, n);
    // a sequence that shrank already has its new length: n_new applies to it once
    if (b < a.B && a.n_new[b] < 0) n = o;
    const int held = pages_of(o, a.shift);
    int need = n > o ? pages_of(n, a.shift) - held : 0;
    long long count = n > o ? n - o : 0;
    const long long pages_to = ask_pages + block_scan(need, warp_sums, &t);
    ask_pages += t;
    const long long toks_to = ask_toks + block_scan(count, warp_sums, &t);
    ask_toks += t;
    if ((need && pages_to > nf) || (count && toks_to > a.tok_cap)) {
      bits |= LLA_STATUS_PAGES_SHORT;
      need = 0;
      count = 0;
      n = o;
    }
    const long long page_at = got_pages + block_scan(need, warp_sums, &t) - need;
    got_pages += t;
    const long long tok_at = got_toks + block_scan(count, warp_sums, &t) - count;
    got_toks += t;
    if (b < a.B) {
      a.tok_start[b] = (int)tok_at;
      if (n > o) a.ctx_len[b] = (int)n;
    }
    for (unsigned m = __ballot_sync(0xffffffffu, need > 0); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const int bb = __shfl_sync(0xffffffffu, b, l), hh = __shfl_sync(0xffffffffu, held, l);
      const int cc = __shfl_sync(0xffffffffu, need, l);
      const long long aa = __shfl_sync(0xffffffffu, page_at, l);
      for (int k = lane; k < cc; k += 32) {
        int page = a.free_list[nf - 1 - (aa + k)];
        if (page < 0 || page >= a.n_pages) {
          bits |= LLA_STATUS_PAGE_RANGE;
          page = -1;
        }
        a.block_table[(long long)bb * a.max_pages + hh + k] = page;
      }
    }
  }
  if (threadIdx.x == 0) {
    a.tok_start[a.B] = (int)got_toks;
    *a.n_free = (int)(nf - got_pages);
  }
  if (bits && a.status) atomicOr(a.status, bits);
  if (a.fill_here) {
    __syncthreads();
    fill_tokens(a, threadIdx.x, kPagesThreads);
  }
}

__global__ void __launch_bounds__(256) pages_fill_kernel(PageMapArgs a) {
  fill_tokens(a, (long long)blockIdx.x * 256 + threadIdx.x, (long long)gridDim.x * 256);
}

}  // namespace

cudaError_t launch_page_map(PageMapArgs a, cudaStream_t s) {
  a.fill_here = a.tok_cap <= 4 * kPagesThreads;
  pages_kernel<<<1, kPagesThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.fill_here) return e;
  const long long blocks = (a.tok_cap + 255) / 256;
  pages_fill_kernel<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lla
