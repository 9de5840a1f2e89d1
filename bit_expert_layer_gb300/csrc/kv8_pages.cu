// kv8_pages.cu -- page tables, offsets, positions and slots of a step, made on the GPU from what
// each sequence keeps and how many tokens it adds.
//
// Sequence b keeps keep[b] positions and adds n_new[b], so it wants after[b] = ceil((keep + new) /
// page_size) pages; it gives back what it holds past that, or takes what it lacks.  Everything
// follows from three sums over the sequences (tokens, pages given, pages taken), which every CTA
// makes for itself in shared memory, so that the CTAs need not wait for one another:
//   token t     the sequence with offsets[b] <= t, position keep[b] + t - offsets[b]
//   page k      taken (in order of sequence and page): of the R pages given the last but k, so
//               that a page changes hands without going through the free list, then the list's
//               own from its end
//   page given  those that are not taken go to the list's end (only where R exceeds the taken
//               ones, so no call both reads and writes the list)
// What a call reads of the state (lengths, pages held, the list's length) it may also have to
// replace, so the CTA that arrives last writes it: by then every other has read it.
// Bound: latency (the launch, the loads of the sequences' numbers, the sums, a page's own loads, the last
// CTA's turn); 8 bytes are written per token.  Measured: a step of 64 sequences, some of which need a
// page and one in nine gives its own back, 5.3 us; 200 prompts of 184 thousand tokens 5.0 us.
#include <algorithm>
#include <cstring>

#include "internal.h"
#include "kv8.cuh"
#include "kv8_host.h"

namespace moe {

namespace {

// 512 threads: 64 tokens over 8 thousand pages 3.7 us, with 1024 4.1, with 256 3.5; a million tokens 7.9,
// 8.2, 10.4; the 8 thousand pages given back at once 9.8, 7.2, 16.7.
constexpr int PG_THREADS = 512, PG_SEQS = KV8_MAX_SEQS, PG_ENTRIES = 8192;

struct PagesParams {
  int* table;
  int* free_pages;
  uint32_t* control;             // error, ticket
  const int *lens, *held, *n_free, *keep, *n_new, *borrowed;
  int *lens_out, *held_out, *n_free_out, *offsets, *positions, *slots;
  int n_seqs, max_pages, n_pages, page_shift, n_tokens, wide;
};

// The last i of 0 .. n - 1 with a[i] <= x (a[0] <= x).
__device__ __forceinline__ int pg_find(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace

__global__ void __launch_bounds__(PG_THREADS) kv8_pages_kernel(const __grid_constant__ PagesParams p) {
  // per sequence: tokens, pages given and taken before it; positions kept (their complement: its tokens get no
  // slots, and nothing is kept), pages held and wanted
  __shared__ int s_off[PG_SEQS + 1], s_give[PG_SEQS + 1], s_take[PG_SEQS + 1];
  __shared__ int s_keep[PG_SEQS], s_held[PG_SEQS], s_rest[PG_SEQS];
  __shared__ int s_warp[PG_THREADS / 32][3];
  __shared__ int s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = p.n_seqs;
  const int cap = p.max_pages << p.page_shift, page = 1 << p.page_shift;
  grid_dep_wait();
  bool bad = false;
  const auto within = [&](int v, int top) {
    const int r = min(max(v, 0), top);
    bad |= r != v;
    return r;
  };
  const int n_free = within(*p.n_free, p.n_pages);
  const int per = (B + PG_THREADS - 1) / PG_THREADS, b0 = min(tid * per, B), b1 = min(b0 + per, B);
  int sum[3] = {0, 0, 0};
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int len = within(p.lens[b], cap), held = within(p.held[b], p.max_pages), fresh = within(p.n_new[b], p.n_tokens);
    const int keep = p.keep ? within(p.keep[b], len) : len;
    const int borrowed = p.borrowed ? within(p.borrowed[b], p.max_pages) : 0;
    // tokens that begin in a borrowed page would go over another sequence's: the sequence is done
    const bool lost = fresh > 0 && keep >> p.page_shift < borrowed;
    bad |= lost || keep + fresh > cap;
    const int after = lost ? 0 : min((keep + fresh + page - 1) >> p.page_shift, p.max_pages);
    const int rest = max(after, borrowed);                   // pages below it are not given back
    s_off[b] = sum[0];
    s_give[b] = sum[1];
    s_take[b] = sum[2];
    s_keep[b] = lost ? ~keep : keep;
    s_held[b] = held;
    s_rest[b] = rest;
    sum[0] += fresh;
    sum[1] += max(held - rest, 0);
    sum[2] += max(after - held, 0);
  }
  int before[3], total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) before[k] = sum[k];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int v = __shfl_up_sync(0xffffffffu, before[k], o);
      if (lane >= o) before[k] += v;
    }
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < 3; ++k) s_warp[warp][k] = before[k];
  __syncthreads();
  // the warps' sums: a lane each
  constexpr int W = PG_THREADS / 32;
  int upto[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) upto[k] = lane < W ? s_warp[lane][k] : 0;
#pragma unroll
  for (int o = 1; o < W; o <<= 1)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int v = __shfl_up_sync(0xffffffffu, upto[k], o);
      if (lane >= o) upto[k] += v;
    }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    total[k] = __shfl_sync(0xffffffffu, upto[k], W - 1);
    const int v = __shfl_sync(0xffffffffu, upto[k], max(warp - 1, 0));
    before[k] += (warp ? v : 0) - sum[k];
  }
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    s_off[b] += before[0];
    s_give[b] += before[1];
    s_take[b] += before[2];
  }
  if (tid == 0) {
    s_off[B] = total[0];
    s_give[B] = total[1];
    s_take[B] = total[2];
  }
  __syncthreads();
  const int given = total[1], wanted = total[2], taken = min(wanted, n_free + given), T = min(total[0], p.n_tokens);
  bad |= wanted > taken || total[0] > p.n_tokens;

  const auto row = [&](int b) { return p.table + static_cast<size_t>(b) * p.max_pages; };
  const auto page_given = [&](int r) {                     // the r-th page given back
    const int b = pg_find(s_give, B, r);
    return row(b)[s_rest[b] + r - s_give[b]];
  };
  const auto page_taken = [&](int k) {
    if (k >= taken) return -1;
    return k < given ? page_given(given - 1 - k) : p.free_pages[n_free - 1 - (k - given)];
  };
  const auto checked = [&](int id) {                       // what changes hands is a page of the pool, or -1
    const bool ok = id >= 0 && id < p.n_pages;
    bad |= !ok;
    return ok ? id : -1;
  };
  const auto page_of = [&](int b, int j) {                 // page j of sequence b, in this step
    if (j >= p.max_pages) return -1;
    return j < s_held[b] ? row(b)[j] : page_taken(s_take[b] + j - s_held[b]);
  };

  const int at = blockIdx.x * PG_THREADS + tid, step = gridDim.x * PG_THREADS;
  // ---- the tables' new entries, -1 where the list ran out
#pragma unroll 1
  for (int k = at; k < wanted; k += step) {
    const int b = pg_find(s_take, B, k);
    row(b)[s_held[b] + k - s_take[b]] = checked(page_taken(k));
  }
  // ---- pages given back and not taken
#pragma unroll 1
  for (int r = at; r < given - taken; r += step) {
    if (n_free + r < p.n_pages) p.free_pages[n_free + r] = checked(page_given(r));
    else bad = true;
  }
  // ---- the tokens, four at a time
#pragma unroll 1
  for (int t0 = 4 * at; t0 < T; t0 += 4 * step) {
    int pos[4], slot[4], b = pg_find(s_off, B, t0), last_b = -1, last_j = -1, id = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + i;
      pos[i] = slot[i] = 0;
      if (t >= T) break;
      while (t >= s_off[b + 1]) ++b;                       // sequences without tokens among them
      const int keep = s_keep[b];
      pos[i] = (keep < 0 ? ~keep : keep) + t - s_off[b];
      const int j = pos[i] >> p.page_shift;
      if (b != last_b || j != last_j) id = keep < 0 ? -1 : page_of(b, j);
      last_b = b;
      last_j = j;
      slot[i] = id < 0 || id >= p.n_pages ? -1 : (id << p.page_shift) + (pos[i] & (page - 1));
      bad |= slot[i] < 0;
    }
    if (p.wide && t0 + 4 <= T) {
      if (p.positions) *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.slots) *reinterpret_cast<int4*>(p.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < T) {
          if (p.positions) p.positions[t0 + i] = pos[i];
          if (p.slots) p.slots[t0 + i] = slot[i];
        }
    }
  }
  if (__syncthreads_or(bad) && tid == 0) atomicOr(p.control, ERRBIT_BOUNDS);
  // ---- the state after the step, by the CTA that arrives last
  if (gridDim.x > 1) {
    if (tid == 0) {
      unsigned old;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p.control + 1) : "memory");
      s_last = old == gridDim.x - 1;
      if (s_last) p.control[1] = 0u;
    }
    __syncthreads();
    if (!s_last) return;
  }
#pragma unroll 1
  for (int b = tid; b <= B; b += PG_THREADS) {
    p.offsets[b] = s_off[b];
    if (b == B) break;
    const int fresh = s_off[b + 1] - s_off[b], len = s_keep[b] < 0 ? 0 : s_keep[b] + fresh;
    const int after = min((len + page - 1) >> p.page_shift, p.max_pages);
    p.lens_out[b] = len;
    p.held_out[b] = min(after, s_held[b] + min(max(taken - s_take[b], 0), s_take[b + 1] - s_take[b]));
  }
  if (tid == 0) *p.n_free_out = min(n_free + given - taken, p.n_pages);
}

}  // namespace moe

using namespace moe;

extern "C" moe_status_t gqa_kv8_pages_step(const gqa_kv8_pages_t* pages, const gqa_kv8_pages_state_t* from,
                                           const gqa_kv8_pages_state_t* to, const int32_t* keep, const int32_t* n_new,
                                           const int32_t* borrowed, int32_t* offsets, int32_t* positions, int32_t* slots,
                                           int n_tokens, moe_stream_t stream) {
  if (!pages || !from || !to || !pages->page_table || !pages->free_pages || !pages->control || !from->lens || !from->held ||
      !from->n_free || !to->lens || !to->held || !to->n_free || !n_new || !offsets)
    return MOE_ERR_INVALID_ARG;
  if (pages->n_seqs < 1 || pages->n_seqs > KV8_MAX_SEQS || pages->max_pages < 1 || pages->n_pages < 1) return MOE_ERR_INVALID_ARG;
  if (pages->page_size < KV8_BLOCK || pages->page_size > 1024 || (pages->page_size & (pages->page_size - 1)))
    return MOE_ERR_INVALID_ARG;
  if (static_cast<long long>(pages->max_pages) * pages->page_size > (1 << 24) ||
      static_cast<long long>(pages->n_pages) * pages->page_size > 0x7FFFFFFFll || n_tokens < 0 || n_tokens > (1 << 20))
    return MOE_ERR_INVALID_ARG;
  const void* all[] = {pages->page_table, pages->free_pages, pages->control, from->lens, from->held, from->n_free, to->lens,
                       to->held, to->n_free, keep, n_new, borrowed, offsets, positions, slots};
  for (const void* x : all)
    if (reinterpret_cast<uintptr_t>(x) & 3u) return MOE_ERR_ALIGNMENT;
  PagesParams p;
  std::memset(&p, 0, sizeof p);
  p.table = pages->page_table;
  p.free_pages = pages->free_pages;
  p.control = pages->control;
  p.lens = from->lens;
  p.held = from->held;
  p.n_free = from->n_free;
  p.keep = keep;
  p.n_new = n_new;
  p.borrowed = borrowed;
  p.lens_out = to->lens;
  p.held_out = to->held;
  p.n_free_out = to->n_free;
  p.offsets = offsets;
  p.positions = positions;
  p.slots = slots;
  p.n_seqs = pages->n_seqs;
  p.max_pages = pages->max_pages;
  p.n_pages = pages->n_pages;
  p.n_tokens = n_tokens;
  while ((1 << p.page_shift) < pages->page_size) ++p.page_shift;
  p.wide = ((reinterpret_cast<uintptr_t>(positions) | reinterpret_cast<uintptr_t>(slots)) & 15u) == 0;
  // A CTA for every 2048 tokens, or for every 8192 pages that may change hands, up to two an SM.  (More
  // for the pages would make most steps, which move few, wait for more CTAs: those 64 tokens 4.4 us with
  // nine CTAs.)
  const long long rows = static_cast<long long>(pages->n_seqs) * pages->max_pages;
  const long long entries = rows < pages->n_pages ? rows : pages->n_pages;
  const long long want = std::max<long long>(n_tokens / (4 * PG_THREADS), entries / PG_ENTRIES) + 1;
  const int grid = static_cast<int>(std::min<long long>(want, 1024 / PG_THREADS * 152));
  const cudaError_t e =
      launch_pdl(kv8_pages_kernel, dim3(grid), dim3(PG_THREADS), 0, reinterpret_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) {
    set_error_detail("gqa_kv8_pages_step: launch", e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

extern "C" moe_status_t gqa_kv8_pages_get_error(const gqa_kv8_pages_t* pages) {
  if (!pages || !pages->control) return MOE_ERR_INVALID_ARG;
  unsigned v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, pages->control, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) e = cudaMemset(pages->control, 0, 4);
  if (e == cudaSuccess && v) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    set_error_detail("gqa_kv8_pages_get_error", e);
    return MOE_ERR_CUDA;
  }
  return v ? MOE_ERR_DEVICE_BOUNDS : MOE_OK;
}
