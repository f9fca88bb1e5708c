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
// pages_kernel (one block, each thread a run of sequences) does the sequences with one
// prefix sum, and the slots of few tokens; many tokens get theirs from pages_fill_kernel.
// Latency is all it costs: a decode step of 256 sequences reads 2 KB and writes 4 KB.
#include "lla_internal.cuh"

namespace lla {
namespace {

__device__ __forceinline__ int pages_of(long long len, int shift) {
  return (int)((len + (1 << shift) - 1) >> shift);
}

// Sums over the block's threads before this one, and of all, of N values at once.
template <int N, int kThreads>
__device__ __forceinline__ void block_scan(const long long (&v)[N], long long (&before)[N],
                                           long long (&total)[N],
                                           long long (*warp_sums)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    before[j] = v[j];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, before[j], o);
      if (lane >= o) before[j] += u;
    }
    if (lane == 31) warp_sums[warp][j] = before[j];
    before[j] -= v[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const long long w = lane < kThreads / 32 ? warp_sums[lane][j] : 0;
    long long all = w, low = lane < warp ? w : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      low += __shfl_xor_sync(0xffffffffu, low, o);
    }
    before[j] += low;
    total[j] = all;
  }
}

// Calls f(l, k) for every thread l and every k < its count, spread over the block's threads:
// each finds its (l, k) in the counts' prefix sums `at` (total in all).
template <int kThreads, typename F>
__device__ __forceinline__ void spread(long long at, long long total, long long* ats, F f) {
  ats[threadIdx.x] = at;
  __syncthreads();
  for (long long i = threadIdx.x; i < total; i += kThreads) {
    int l = 0;
#pragma unroll
    for (int w = kThreads / 2; w > 0; w >>= 1)
      if (ats[l + w] <= i) l += w;
    f(l, (int)(i - ats[l]));
  }
  __syncthreads();
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) pages_kernel(PageMapArgs a) {
  __shared__ long long sums3[kThreads / 32][3], sums2[kThreads / 32][2];
  __shared__ long long ats[kThreads];
  __shared__ long long froms[kThreads], sums1[kThreads / 32][1];
  __shared__ int at_b[kThreads], at_row[kThreads];
  const long long limit = (long long)a.max_pages << a.shift;
  const int per = (a.B + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
  int nf = *a.n_free;
  int bits = 0;
  if (nf < 0 || nf > a.n_pages) {
    bits |= LLA_STATUS_PAGE_RANGE;
    nf = nf < 0 ? 0 : a.n_pages;
  }

  // length of sequence b before and after; a length outside its table is left alone
  struct Grow {
    int old_len, new_len;
  };
  auto lengths = [&](int b) {
    Grow g{0, 0};
    if (b >= a.B) return g;
    g.old_len = g.new_len = a.ctx_len[b];
    if (g.old_len < 0 || g.old_len > limit) {
      bits |= LLA_STATUS_CTX_RANGE;
      return g;
    }
    const long long to = (long long)g.old_len + a.n_new[b];
    if (to > limit) {
      bits |= LLA_STATUS_CTX_RANGE;
      return g;
    }
    g.new_len = to < 0 ? 0 : (int)to;
    return g;
  };
  auto need_of = [&](const Grow& g) {
    return g.new_len > g.old_len ? pages_of(g.new_len, a.shift) - pages_of(g.old_len, a.shift) : 0;
  };

  // pages given back, pages and tokens asked for
  long long v[3] = {0, 0, 0}, before[3], total[3];
  bool shrinks = false;
  for (int k = 0; k < per; ++k) {
    const Grow g = lengths(b0 + k);
    if (g.new_len < g.old_len) {
      shrinks = true;
      v[0] += pages_of(g.old_len, a.shift) - pages_of(g.new_len, a.shift);
    } else {
      v[1] += need_of(g);
      v[2] += g.new_len - g.old_len;
    }
  }
  block_scan<3, kThreads>(v, before, total, sums3);

  // Each of a thread's sequences in turn, all threads' together.
  if (__syncthreads_or(shrinks)) {
    const long long gone = total[0];
    long long at = before[0];
    for (int k = 0; k < per; ++k) {
      const int b = b0 + k;
      const Grow g = lengths(b);
      const bool cut = g.new_len < g.old_len;
      const int first = pages_of(g.new_len, a.shift);
      const int back = cut ? pages_of(g.old_len, a.shift) - first : 0;
      at_b[threadIdx.x] = b;
      at_row[threadIdx.x] = first;
      froms[threadIdx.x] = at;
      long long part[1] = {back}, lead[1], all[1] = {total[0]};
      lead[0] = at;
      if (per > 1) block_scan<1, kThreads>(part, lead, all, sums1);
      spread<kThreads>(lead[0], all[0], ats, [&](int l, int i) {
        int32_t* entry = a.block_table + (long long)at_b[l] * a.max_pages + at_row[l] + i;
        int page = *entry;
        *entry = -1;
        if (page < 0 || page >= a.n_pages) {
          bits |= LLA_STATUS_PAGE_RANGE;
          page = -1;
        }
        const long long to = nf + gone - 1 - (froms[l] + i);    // pushed in reverse
        if (to < a.n_pages) a.free_list[to] = page;
        else bits |= LLA_STATUS_PAGE_RANGE;
      });
      at += back;
      if (cut) a.ctx_len[b] = g.new_len;
    }
    nf = (int)(nf + gone < a.n_pages ? nf + gone : a.n_pages);
    __syncthreads();
  }

  // Growing sequences, in order: served while everything asked so far fits.  A sequence
  // that shrank has its new length already; n_new applies to it once.
  auto grows = [&](int b) {
    Grow g{0, 0};
    if (b < a.B && a.n_new[b] > 0) g = lengths(b);
    return g;
  };
  auto fits = [&](const Grow& g, long long pages_to, long long toks_to) {
    return (need_of(g) == 0 || pages_to <= nf) && (g.new_len == g.old_len || toks_to <= a.tok_cap);
  };
  long long got[2] = {0, 0}, got_before[2] = {before[1], before[2]}, got_total[2] = {total[1], total[2]};
  bool refused = false;
  if (total[1] > nf || total[2] > a.tok_cap) {                  // block-uniform
    long long pages_to = before[1], toks_to = before[2];
    for (int k = 0; k < per; ++k) {
      const Grow g = grows(b0 + k);
      pages_to += need_of(g);
      toks_to += g.new_len - g.old_len;
      if (fits(g, pages_to, toks_to)) {
        got[0] += need_of(g);
        got[1] += g.new_len - g.old_len;
      } else {
        bits |= LLA_STATUS_PAGES_SHORT;
      }
    }
    refused = true;
    block_scan<2, kThreads>(got, got_before, got_total, sums2);
  }
  long long pages_to = before[1], toks_to = before[2];
  long long page_at = got_before[0], tok_at = got_before[1];
  for (int k = 0; k < per; ++k) {
    const int b = b0 + k;
    Grow g = grows(b);
    if (refused) {
      pages_to += need_of(g);
      toks_to += g.new_len - g.old_len;
      if (!fits(g, pages_to, toks_to)) g.new_len = g.old_len;
    }
    const int held = pages_of(g.old_len, a.shift), need = need_of(g), count = g.new_len - g.old_len;
    if (b < a.B) {
      a.tok_start[b] = (int)tok_at;
      if (count) a.ctx_len[b] = g.new_len;
    }
    at_b[threadIdx.x] = b;
    at_row[threadIdx.x] = held;
    froms[threadIdx.x] = page_at;
    long long part[2] = {need, count}, lead[2] = {page_at, tok_at};
    long long all[2] = {got_total[0], got_total[1]};
    if (per > 1) {
      __syncthreads();                                          // sums2 has been read
      block_scan<2, kThreads>(part, lead, all, sums2);
    }
    spread<kThreads>(lead[0], all[0], ats, [&](int l, int i) {
      int page = a.free_list[nf - 1 - (froms[l] + i)];
      if (page < 0 || page >= a.n_pages) {
        bits |= LLA_STATUS_PAGE_RANGE;
        page = -1;
      }
      a.block_table[(long long)at_b[l] * a.max_pages + at_row[l] + i] = page;
    });
    if (a.fill_here) {                                          // the table's entries are there
      at_row[threadIdx.x] = g.old_len;
      froms[threadIdx.x] = tok_at;
      spread<kThreads>(lead[1], all[1], ats, [&](int l, int i) {
        const int pos = at_row[l] + i;
        const int page = a.block_table[(long long)at_b[l] * a.max_pages + (pos >> a.shift)];
        const bool known = page >= 0 && page < a.n_pages;
        if (!known) bits |= LLA_STATUS_PAGE_RANGE;
        const long long to = froms[l] + i;
        a.slot[to] = known ? ((long long)page << a.shift) + (pos & ((1 << a.shift) - 1)) : -1;
        a.positions[to] = pos;
      });
    }
    page_at += need;
    tok_at += count;
  }
  if (a.fill_here)
    for (long long i = got_total[1] + threadIdx.x; i < a.tok_cap; i += kThreads) {
      a.slot[i] = -1;
      a.positions[i] = 0;
    }
  if (threadIdx.x == 0) {
    a.tok_start[a.B] = (int)got_total[1];
    *a.n_free = (int)(nf - got_total[0]);
  }
  if (bits && a.status) atomicOr(a.status, bits);
}

// Slots and positions, one token per thread.
__global__ void __launch_bounds__(256) pages_fill_kernel(PageMapArgs a) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.tok_cap) return;
  if (i >= a.tok_start[a.B]) {
    a.slot[i] = -1;
    a.positions[i] = 0;
    return;
  }
  int lo = 0, hi = a.B;                         // tok_start[lo] <= i < tok_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.tok_start[mid] <= i) lo = mid;
    else hi = mid;
  }
  const int pos = a.ctx_len[lo] - (a.tok_start[lo + 1] - (int)i);
  const int page = a.block_table[(long long)lo * a.max_pages + (pos >> a.shift)];
  const bool known = page >= 0 && page < a.n_pages;
  if (!known && a.status) atomicOr(a.status, LLA_STATUS_PAGE_RANGE);
  a.slot[i] = known ? ((long long)page << a.shift) + (pos & ((1 << a.shift) - 1)) : -1;
  a.positions[i] = pos;
}

}  // namespace

cudaError_t launch_page_map(PageMapArgs a, cudaStream_t s) {
  // One block writes 4096 tokens in the time that a second launch takes.
  a.fill_here = a.tok_cap <= 4096;
  // 256 threads meet faster than 1024, which write the pages of prompts faster.
  if (a.B <= 256 && a.fill_here)
    pages_kernel<256><<<1, 256, 0, s>>>(a);
  else
    pages_kernel<1024><<<1, 1024, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.fill_here) return e;
  pages_fill_kernel<<<(unsigned)((a.tok_cap + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lla
