// kv8_sched.cuh -- how the attention kernels over the 8-bit cache share their work.
//
// A tile is TQ consecutive new tokens of one sequence for one key/value head: TQ * G query
// rows that read the same keys.  Its work is cut into units of U positions, as many as the
// tile's last token sees.  All tiles' units form one line, ordered by sequence, head and
// tile, and every worker (a CTA, or a warp of it) takes an equal run of the line, so the
// load is even whatever the lengths are and the lengths can stay on the device.  A run holds
// whole tiles and at most one part at either end.  The parts of a tile meet first inside
// the CTA, then through the workspace: each CTA leaves its unnormalised sums in a slot of
// its own (2 per CTA: a tile that began before the CTA's runs, a tile that goes on after
// them), to be added up in the order of the line: in the decode kernel by the last CTA to
// arrive, by a ticket that belongs to the tile's first CTA, for prompts by a second kernel.
// Nothing waits.
//
// Nothing is tabulated per tile: a sequence's units up to tile t have a closed form.  With
// TQ a power of two that divides U, r = U / TQ, `a` the first new token's position and
// A = (a + U - 1) / TQ, tile i sees a + TQ (i + 1) positions, which is (A + i + 1) / r units
// (whole divisions; the last tile sees all of the sequence), and the sum of x / r over
// x = 0 .. X is r q (q - 1) / 2 + q (m + 1) with q = X / r, m = X mod r.  With TQ = c U it is
// (a + U - 1) / U + c (i + 1) units.
// Starting a tile costs as much as some units (its queries are fetched, its result written),
// so each has C more units in the line than positions to see; they come first, and a run
// that ends inside them leaves the tile to the next.
#pragma once

#include "kv8.cuh"

namespace moe {

constexpr int KV8_MAX_CTAS = 160;
constexpr int KV8_MAX_DEVICES = 64;
constexpr int KV8_TICKET_BYTES = 1024;   // the workspace's first bytes: one ticket per CTA
// A query row is brought to [2^13, 2^14) by 2^-e, e within these bounds (any finite bf16 row fits
// fp16 then, and 2^e times a score scale of ordinary size is a normal number).  The factor
// of its scores, 2^e times the score scale times the keys' scale, ends at the last: past it the
// scores themselves leave fp32, and a score of zero stays one.
constexpr int KV8_Q_MIN_EXP = -120, KV8_Q_MAX_EXP = 115;
constexpr float KV8_MAX_FACTOR = 0x1p126f;
// A row's references: ms, the largest score so far, and d.  Its weights are
//   w_i = 2^(s_i - ms + e_i - d), 2^e_i being the scale of the value's block,
// and its normaliser is sum_i 2^(s_i - ms), which must not carry the scales: blocks of zeros
// have the smallest one there is, 2^-100, and in units of the weights their share of the
// normaliser passes fp32 after some thousand positions.  A term of the normaliser is
// w_i 2^(d - e_i) as long as that exponent is at most KV8_SUM_TOP, so that terms stay under
// 2^80 and 2^24 of them in range; else the references move first, and the terms are
// exponentials of their own.
constexpr float KV8_SUM_TOP = 64.0f;
// Scores are products rounded once with the references in one multiply-add.  Past KV8_FAR the
// part of the product that rounding would have cut off is itself worth powers of two, so that
// there, and where no score has been seen yet, the score is rounded first.  One past fp32's
// range counts as its largest number.
constexpr float KV8_FAR = 0x1p20f;
constexpr float KV8_NO_REF = -0x1.fffffep127f;
__device__ __forceinline__ float kv8_end(float s) {      // NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(s), "f"(KV8_NO_REF));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(-KV8_NO_REF));
  return r;
}
// The value product takes the weights in fp16, which holds 11 bits of them from 2^-14 to 2^16.
// Where the references move, the largest weight of the positions at hand becomes 2^KV8_W_FIRST; they
// move again when one passes 2^KV8_W_TOP, and also when the largest is below a bound (LOW: chosen
// by the kernels, so that what subnormal weights lose, 2^-25 each, is under 2^-11 of the largest
// one of theirs).  Without the latter a single position with nearly all the weight (and, as such
// positions have it, a value near zero) would cost the others their bits: 32 thousand positions
// with 0.1 % of the weight came out 33 % off.  A row's unit comes no further down than
// 2^-KV8_W_SPAN of its highest, which keeps sums in fp32's range, so that weights under that of
// the largest are lost, nor under 2^KV8_W_LEAST.  (First 9 or 11: 470 and 475 us for a piece of a
// prompt that takes 408 with 7, from the moves.)
constexpr float KV8_W_FIRST = 7.0f, KV8_W_TOP = 15.0f, KV8_W_SPAN = 40.0f, KV8_W_LEAST = -118.0f;
constexpr float KV8_W_LOST = KV8_W_FIRST - KV8_W_SPAN;
// Whether d comes down from `was`, for positions whose largest weight is 2^top in units of ms.
__device__ __forceinline__ bool kv8_down(float top, float was, float low, float ms, float peak) {
  const float to = top - KV8_W_FIRST;
  return top < was + low && to > fmaxf(peak - ms - KV8_W_SPAN, KV8_W_LEAST) && fabsf(ms) < KV8_FAR;
}

struct Kv8AttnParams {
  Kv8Cache c;
  Kv8Batch b;
  const __nv_bfloat16* q;
  long long q_stride;
  __nv_bfloat16* out;
  int hq, G, tq_shift;
  float scale_log2;      // score scale * log2(e)
  int out_wide;          // out is 32-byte aligned
  unsigned* tickets;     // [KV8_MAX_CTAS], zero between calls
  float* part;           // [CTA][2][rows][row floats]
  unsigned long long wait_ns;
};

// A run of units inside one tile.
struct Kv8Seg {
  Kv8Seq s;
  int b, g, t;           // sequence, key/value head, tile of the sequence
  int u0, u1, units;     // this run's units of positions (none: u1 <= u0), the tile's
  int len;               // units of the line that the segment takes
  int x;                 // units of the line before it in its tile
};

// The line cut into n runs: run i is units i total / n up to (i + 1) total / n, and unit w
// belongs to run ((w + 1) n - 1) / total (whole divisions).
struct Kv8Runs {
  long long total;
  int n;
};
// Code that is fetched once per launch costs more than its arithmetic (some 250 cycles per 8
// instructions that come from L2), so the rare long division is a function of its own.
static __device__ __noinline__ long long kv8_div_long(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long kv8_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return kv8_div_long(a, b);
}
__device__ __forceinline__ long long kv8_run_begin(const Kv8Runs& r, int i) { return kv8_div(i * r.total, r.n); }
__device__ __forceinline__ int kv8_run_of(const Kv8Runs& r, long long w) {
  return static_cast<int>(kv8_div((w + 1) * r.n - 1, r.total));
}

__device__ __forceinline__ long long kv8_upto(long long x, int r_shift) {
  const long long q = x >> r_shift, m = x & ((1ll << r_shift) - 1);
  return ((q * (q - 1)) << r_shift) / 2 + q * (m + 1);
}

// Units of tiles 0 .. t - 1 of a sequence (t at most its last tile).
template <int U, int C>
__device__ __forceinline__ long long kv8_units_before(const Kv8Seq& s, int tq_shift, int t) {
  constexpr int US = U == 16 ? 4 : U == 32 ? 5 : U == 64 ? 6 : 7;
  static_assert((1 << US) == U, "U is 16 to 128");
  const long long n = t;
  if (tq_shift > US) return n * ((max(s.first, 0) + U - 1) / U + C) + ((n * (n + 1) / 2) << (tq_shift - US));
  const int rs = US - tq_shift;
  const long long A = (max(s.first, 0) + U - 1) >> tq_shift;
  return kv8_upto(A + t, rs) - kv8_upto(A, rs) + C * n;
}
// Units of one tile: what its last token sees, one at least, and C.
template <int U, int C>
__device__ __forceinline__ int kv8_units_tile(const Kv8Seq& s, int tq_shift, int t) {
  return (max(s.first, 0) + min((t + 1) << tq_shift, s.n) + U - 1) / U + C;
}
template <int U, int C>
__device__ __forceinline__ long long kv8_units_seq(const Kv8Seq& s, int tq_shift) {
  if (s.n <= 0) return 0;
  if (s.n <= (1 << tq_shift)) return kv8_units_tile<U, C>(s, tq_shift, 0);
  const int tiles = (s.n + (1 << tq_shift) - 1) >> tq_shift;
  return kv8_units_before<U, C>(s, tq_shift, tiles - 1) + kv8_units_tile<U, C>(s, tq_shift, tiles - 1);
}

// The line: prefix[b] = units before sequence b (all heads), in shared memory, filled by
// the whole CTA (THREADS threads, s_warp: THREADS / 32 words); returns its length.
template <int U, int C, int THREADS>
__device__ __forceinline__ long long kv8_line(const Kv8AttnParams& p, long long* prefix, long long* s_warp) {
  const int tid = threadIdx.x, B = p.b.n_seqs;
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long sum = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Kv8Seq s = kv8_seq(p.b, p.c.page_shift, b);
    // (fewer positions than new tokens: the tokens without one get zeros)
    if ((s.bad || (s.n > 0 && s.first < 0)) && blockIdx.x == 0) atomicOr(p.c.err, ERRBIT_BOUNDS);
    sum += kv8_units_seq<U, C>(s, p.tq_shift) * p.c.hkv;
    prefix[b] = sum;                       // inside this thread's run for now
  }
  long long incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if ((tid & 31) >= o) incl += v;
  }
  if ((tid & 31) == 31) s_warp[tid >> 5] = incl;
  __syncthreads();
  long long before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long v = s_warp[w];
    if (w < (tid >> 5)) before += v;
    total += v;
  }
  // exclusive: prefix[b] = everything before b
  long long prev = before;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const long long incl_b = before + prefix[b];
    prefix[b] = prev;
    prev = incl_b;
  }
  if (tid == 0) prefix[B] = total;
  __syncthreads();
  return total;
}

// Ends the segment that starts at unit w, x units into its tile of `all` units, with the tile or
// at w_end.
template <int C>
__device__ __forceinline__ void kv8_seg_close(Kv8Seg& g, int x, int all, long long w, long long w_end) {
  const long long left = w_end - w;
  const int end = all - x <= left ? all : x + static_cast<int>(left);
  g.x = x;
  g.len = end - x;
  g.units = all - C;
  g.u0 = max(x - C, 0);
  g.u1 = end - C;
}
// The runs that hold the first and the last unit of positions of the segment's tile (the
// segment starts at unit w).
template <int C>
__device__ __forceinline__ int2 kv8_owners(const Kv8Seg& g, long long w, const Kv8Runs& runs) {
  const long long start = w - g.x;
  return make_int2(kv8_run_of(runs, start + C), kv8_run_of(runs, start + C + g.units - 1));
}

// The last of 0 .. n - 1 that satisfies `ok`, which holds up to some point and not after it, and
// for 0: a search by the whole (converged) warp, 32 ways a step.
template <typename F>
__device__ __forceinline__ int kv8_last_of(int n, F ok) {
  const int lane = lane_id();
  int lo = 0;
#pragma unroll 1
  while (n > 1) {
    const int step = (n + 31) / 32, i = lane * step;
    const bool in = i < n && (lane == 0 || ok(lo + i));
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, in));
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

// The segment that starts at unit w of the line (asked for by whole warps).
template <int U, int C>
__device__ __forceinline__ Kv8Seg kv8_seg(const Kv8AttnParams& p, const long long* prefix, long long w,
                                          long long w_end) {
  Kv8Seg g;
  const int lo = kv8_last_of(p.b.n_seqs, [&](int i) { return prefix[i] <= w; });
  g.b = lo;
  g.s = kv8_seq(p.b, p.c.page_shift, lo);
  long long x = w - prefix[lo];
  const long long per_head = kv8_units_seq<U, C>(g.s, p.tq_shift);
  g.g = 0;
  if (p.c.hkv > 4) {
    g.g = static_cast<int>(kv8_div(x, per_head));
    x -= g.g * per_head;
  } else {
#pragma unroll 1
    for (; x >= per_head; x -= per_head) ++g.g;
  }
  const int tiles = (g.s.n + (1 << p.tq_shift) - 1) >> p.tq_shift;
  const int tl = kv8_last_of(tiles, [&](int t) { return kv8_units_before<U, C>(g.s, p.tq_shift, t) <= x; });
  g.t = tl;
  const int in_tile = static_cast<int>(tl ? x - kv8_units_before<U, C>(g.s, p.tq_shift, tl) : x);
  kv8_seg_close<C>(g, in_tile, kv8_units_tile<U, C>(g.s, p.tq_shift, tl), w, w_end);
  return g;
}

// The segment after `g`, at unit w of the line (g was not the run's last): it begins a tile,
// the sequence's next one, or the first of the next head or sequence.
template <int U, int C>
__device__ __forceinline__ void kv8_next(Kv8Seg& g, const Kv8AttnParams& p, const long long* prefix, long long w,
                                         long long w_end) {
  const int tiles = (g.s.n + (1 << p.tq_shift) - 1) >> p.tq_shift;
  if (++g.t >= tiles) {
    g.t = 0;
    if (++g.g >= p.c.hkv) {
      g.g = 0;
      do ++g.b; while (prefix[g.b + 1] <= w);      // sequences without new tokens have no units
      g.s = kv8_seq(p.b, p.c.page_shift, g.b);
    }
  }
  kv8_seg_close<C>(g, 0, kv8_units_tile<U, C>(g.s, p.tq_shift, g.t), w, w_end);
}

// Positions that the tile's last token sees.  (The tile's units are counted as if the sequence
// began at position 0 at the latest, so that with fewer positions than new tokens, first < 0, the
// last units lie past this.)
__device__ __forceinline__ int kv8_seg_end(const Kv8Seg& g, int tq_shift) {
  return max(g.s.first + min((g.t + 1) << tq_shift, g.s.n), 0);
}

}  // namespace moe
