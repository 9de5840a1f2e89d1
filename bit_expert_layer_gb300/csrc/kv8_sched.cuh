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
//
// The four modes differ in the positions that a tile's units stand for:
//   causal   0 up to the tile's last token
//   window   the granules (of 16 positions for prompts, 32 for decode) that the first `sinks` touch,
//            then those of the windows of the tile's tokens, one after the other as if the ones
//            between them were not there; units are cut from that row.  The line counts a tile's
//            units by a bound that needs no search, the causal count or K = kv8_win_units(),
//            whichever is less; what a tile has less than that are units without positions at its
//            end, which no run works on.
//   prefix   the line's items are groups of sequences, an item's tokens those of all of the group's
//            sequences, and every token sees all of the group's shared positions
//   suffix   causal, from the first position on that the prefix pass left
#pragma once

#include "kv8.cuh"

namespace moe {

constexpr int KV8_MAX_CTAS = 160;
constexpr int KV8_MAX_DEVICES = 64;
constexpr int KV8_TICKET_BYTES = 1024;   // the workspace's first bytes: one ticket per CTA
enum Kv8Mode { KV8_CAUSAL, KV8_WINDOW, KV8_PREFIX, KV8_SUFFIX };
// Whether a kernel's runs may be aligned to tiles (see kv8_line): prompts with a window.
__host__ __device__ constexpr bool kv8_aligns(int U, int mode) { return U == 128 && mode == KV8_WINDOW; }
__host__ __device__ constexpr int kv8_granule(int U) { return U == 128 ? 16 : U; }
// Shared positions are worked on in whole units of either kernel; a sequence sees to the rest itself.
constexpr int KV8_SHARED_UNIT = 128;
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
  int window, sinks;     // window mode: positions of a window, first positions that stay visible
  int win_units;         // and the most units that a tile has there
  const int* groups;     // prefix and suffix modes: first sequence of each group, the end
  const int* shared;     // positions that each group shares
  int n_groups, max_shared;
  float* rows;           // sums of the query rows, [token][query head][kv8_row_floats(D)]: what the prefix pass leaves,
  float* own;            // and in side-by-side passes what the suffix pass leaves (else null)
  int shift_prefix, shift_suffix;   // side by side: tokens of the two passes' tiles, as shifts
};

// (see kv8_split)
constexpr float KV8_SPLIT_SUFFIX = 11.0f, KV8_SPLIT_PREFIX = 11.0f, KV8_SPLIT_ROWS8 = 0.18f, KV8_SPLIT_ROWS16 = 0.27f,
                KV8_SPLIT_ONE = 1.3f, KV8_SPLIT_TWO = 1.95f;

// Workspace of a query row's sums (O, references ms and d, normaliser): 32-byte rows.
__host__ __device__ constexpr int kv8_row_floats(int D) { return D + 8; }

// Two sums of one row with references of their own become one: its normaliser, the factors of the
// two O, and the unit of the result's weights in the normaliser's.
struct Kv8Join {
  float sum, f[2], unit;
};
__device__ __forceinline__ Kv8Join kv8_join(const float4& a, const float4& b) {    // each {ms, d, normaliser}
  Kv8Join j;
  const float m = fmaxf(a.x, b.x), da = a.x - m + a.y, db = b.x - m + b.y, top = fmaxf(da, db);
  j.sum = fmaf(ex2(a.x - m), a.z, ex2(b.x - m) * b.z);
  j.f[0] = ex2(da - top);
  j.f[1] = ex2(db - top);
  j.unit = ex2(top);
  return j;
}

// Window mode: the most units of a tile, by the granules that W + TQ - 1 consecutive positions can
// touch and the sinks'.
__host__ __device__ constexpr int kv8_win_units(int U, int tq, int window, int sinks) {
  const int g = kv8_granule(U);
  return (((window + tq - 1 + 2 * g - 2) / g + (sinks + g - 1) / g) * g + U - 1) / U;
}

// A run of units inside one tile.
struct Kv8Seg {
  Kv8Seq s;
  int b, g, t;           // sequence, key/value head, tile of the sequence
  int u0, u1, units;     // this run's units of positions (none: u1 <= u0), the tile's
  int len;               // units of the line that the segment takes
  int x;                 // units of the line before it in its tile
  int sunk, skip;        // window mode: positions of the sinks' granules, and positions left out after them
  int low;               // and the first position of the window of the tile's first token
};
// Where positions of a segment's tile stand: place i of its row (unit u begins at place u U) is position
// i + kv8_skip(i).
template <int MODE>
__device__ __forceinline__ int kv8_skip(const Kv8Seg& g, int i) {
  if constexpr (MODE == KV8_WINDOW) return i < g.sunk ? 0 : g.skip;
  if constexpr (MODE == KV8_SUFFIX) return g.s.base;
  return 0;
}

// The line cut into n runs: run i is units i span / n up to (i + 1) span / n, and unit w
// belongs to run ((w + 1) n - 1) / span (whole divisions).  The span is the line's length, or for
// prompts with a window a little more, so that runs begin where tiles do: see kv8_line.
struct Kv8Runs {
  long long total, span;
  int n;
};
// The line as it lies in shared memory: units before each item; in suffix mode what the prefix pass
// has seen to of each sequence (in window mode, while the line is made, tiles); and the length
// that every tile counts with, where it is one.
struct Kv8Line {
  long long* prefix;
  int* base;
  int uni;
  bool shares;           // prefix and suffix mode: groups and sequences are in order
};
// Code that is fetched once per launch costs more than its arithmetic (some 250 cycles per 8
// instructions that come from L2), so the rare long division is a function of its own.
static __device__ __noinline__ long long kv8_div_long(long long a, long long b) { return a / b; }
__device__ __forceinline__ long long kv8_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return kv8_div_long(a, b);
}
template <int U, int MODE>
__device__ __forceinline__ long long kv8_run_begin(const Kv8Runs& r, int i) {
  if constexpr (kv8_aligns(U, MODE)) return min(kv8_div(i * r.span, r.n), r.total);
  return kv8_div(i * r.total, r.n);
}
template <int U, int MODE>
__device__ __forceinline__ int kv8_run_of(const Kv8Runs& r, long long w) {
  return static_cast<int>(kv8_div((w + 1) * r.n - 1, kv8_aligns(U, MODE) ? r.span : r.total));
}

__device__ __forceinline__ long long kv8_upto(long long x, int r_shift) {
  const long long q = x >> r_shift, m = x & ((1ll << r_shift) - 1);
  return ((q * (q - 1)) << r_shift) / 2 + q * (m + 1);
}

// The position that the tiles' units are counted from: the first new token's, less what a prefix
// pass has done.
template <int MODE>
__device__ __forceinline__ int kv8_from(const Kv8Seq& s) {
  return max(s.first, 0) - (MODE == KV8_SUFFIX ? s.base : 0);
}
// Units of tiles 0 .. t - 1 of a sequence (t at most its last tile).
template <int U, int C, int MODE>
__device__ __forceinline__ long long kv8_units_before(const Kv8AttnParams& p, int uni, const Kv8Seq& s, int t) {
  if (kv8_aligns(U, MODE) && uni) return static_cast<long long>(t) * uni;
  constexpr int US = U == 16 ? 4 : U == 32 ? 5 : U == 64 ? 6 : 7;
  static_assert((1 << US) == U, "U is 16 to 128");
  const int from = kv8_from<MODE>(s), tq_shift = p.tq_shift;
  long long n = t, rest = 0;
  if constexpr (MODE == KV8_PREFIX) return n * (s.len / U + C);
  if constexpr (MODE == KV8_WINDOW) {
    // tile i has K = win_units or more by the causal count from i + 1 >= ((K - 1) U + 1 - from) / TQ on
    const int full = max(((p.win_units - 1) * U - from) >> tq_shift, 0);
    if (t > full) {
      rest = static_cast<long long>(t - full) * (p.win_units + C);
      n = full;
    }
  }
  if (tq_shift > US) return rest + n * ((from + U - 1) / U + C) + ((n * (n + 1) / 2) << (tq_shift - US));
  const int rs = US - tq_shift;
  const long long A = (from + U - 1) >> tq_shift;
  return rest + kv8_upto(A + n, rs) - kv8_upto(A, rs) + C * n;
}
// Units of one tile: what its last token sees, one at least, and C.
template <int U, int C, int MODE>
__device__ __forceinline__ int kv8_units_tile(const Kv8AttnParams& p, int uni, const Kv8Seq& s, int t) {
  if (kv8_aligns(U, MODE) && uni) return uni;
  if constexpr (MODE == KV8_PREFIX) return s.len / U + C;
  const int n = (kv8_from<MODE>(s) + min((t + 1) << p.tq_shift, s.n) + U - 1) / U;
  return (MODE == KV8_WINDOW ? min(n, p.win_units) : n) + C;
}
template <int U, int C, int MODE>
__device__ __forceinline__ long long kv8_units_seq(const Kv8AttnParams& p, int uni, const Kv8Seq& s) {
  if (s.n <= 0) return 0;
  if (s.n <= (1 << p.tq_shift)) return kv8_units_tile<U, C, MODE>(p, uni, s, 0);
  const int tiles = (s.n + (1 << p.tq_shift) - 1) >> p.tq_shift;
  return kv8_units_before<U, C, MODE>(p, uni, s, tiles - 1) + kv8_units_tile<U, C, MODE>(p, uni, s, tiles - 1);
}

// The positions of a group that the prefix pass works on, of the `shared` that it says it shares; `fits` when
// the page table holds those.
__device__ __forceinline__ int kv8_group_len(const Kv8AttnParams& p, int shared, bool* fits) {
  const int len = min(max(shared, 0), p.b.max_pages << p.c.page_shift);
  *fits = len == shared;
  return min(len, p.max_shared) / KV8_SHARED_UNIT * KV8_SHARED_UNIT;
}
// A group of sequences with a shared prefix as an item of the line: the tokens of all of them,
// each seeing `len` positions (whole units).  `bad` when something was out of range.
__device__ __forceinline__ Kv8Seq kv8_group(const Kv8AttnParams& p, int i) {
  Kv8Seq s;
  // (kept to the batch here; kv8_line finds out whether they were)
  const int b0 = min(max(__ldg(p.groups + i), 0), p.b.n_seqs), b1 = min(max(__ldg(p.groups + i + 1), 0), p.b.n_seqs);
  const int shared = __ldg(p.shared + i);
  const int o0 = __ldg(p.b.offsets + b0), o1 = __ldg(p.b.offsets + b1);
  const bool rows = o0 >= 0 && o0 <= o1 && o1 <= p.b.n_tokens;
  bool fits;
  s.off = rows ? o0 : 0;
  s.len = kv8_group_len(p, shared, &fits);
  s.n = rows && s.len > 0 ? o1 - o0 : 0;
  s.first = 0;
  s.base = 0;
  s.bad = !rows || !fits;
  return s;
}
// The positions of sequence b that the prefix pass sees to: those of its group, if all of its new
// tokens come after them.  (Where that counts, kv8_line has found every sequence's rows in order, so that
// the group's are those of its sequences.)
__device__ __forceinline__ int kv8_base(const Kv8AttnParams& p, const Kv8Seq& s, int b) {
  int lo = 0, hi = p.n_groups;           // the last group that begins at b or before
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.groups + mid) <= b) lo = mid;
    else hi = mid;
  }
  const int g0 = __ldg(p.groups + lo), g1 = __ldg(p.groups + lo + 1), shared = __ldg(p.shared + lo);
  bool fits;
  const int len = kv8_group_len(p, shared, &fits);
  return s.n > 0 && b >= g0 && b < g1 && s.first >= len ? len : 0;
}
// Item i of the line: a sequence, or in prefix mode a group.  (base: filled by kv8_line.)
template <int MODE>
__device__ __forceinline__ Kv8Seq kv8_item(const Kv8AttnParams& p, const int* base, int i) {
  if constexpr (MODE == KV8_PREFIX) {
    return kv8_group(p, i);
  } else {
    Kv8Seq s = kv8_seq(p.b, p.c.page_shift, i);
    s.base = MODE == KV8_SUFFIX ? base[i] : 0;
    return s;
  }
}
template <int MODE>
__device__ __forceinline__ int kv8_items(const Kv8AttnParams& p) { return MODE == KV8_PREFIX ? p.n_groups : p.b.n_seqs; }
// The page-table row of item i.
template <int MODE>
__device__ __forceinline__ const int* kv8_table(const Kv8AttnParams& p, int i) {
  const int b = MODE == KV8_PREFIX ? __ldg(p.groups + i) : i;
  return p.b.page_table + static_cast<size_t>(b) * p.b.max_pages;
}

// How many of `grid` CTAs the suffix pass gets where the two passes run side by side: those under
// which the longer of the two is shortest.  units, pieces: the prefix pass's units (of one or two
// row blocks) and the suffix pass's pieces (of 8 or 16 query rows).  The constants are microseconds, measured with 128
// sequences over 32768 shared positions: what a CTA takes for one, and before and after them.
__device__ __forceinline__ int kv8_split(long long units, long long pieces, bool one_block, bool rows8, int grid) {
  if (units <= 0) return grid;
  const float u = static_cast<float>(units) * (one_block ? KV8_SPLIT_ONE : KV8_SPLIT_TWO);
  const float s = static_cast<float>(pieces) * (rows8 ? KV8_SPLIT_ROWS8 : KV8_SPLIT_ROWS16);
  float best = INFINITY;
  int at = 1;
#pragma unroll 1
  for (int i = lane_id() + 1; i < grid; i += 32) {
    const float t = fmaxf(KV8_SPLIT_SUFFIX + __fdividef(s, i), KV8_SPLIT_PREFIX + __fdividef(u, grid - i));
    if (t < best) {
      best = t;
      at = i;
    }
  }
#pragma unroll 1
  for (int o = 16; o >= 1; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, best, o);
    const int i = __shfl_xor_sync(0xffffffffu, at, o);
    if (t < best || (t == best && i < at)) {
      best = t;
      at = i;
    }
  }
  return at;
}

// A sequence's share of the suffix pass's pieces, from position `from` of its own on.  A tile counts
// eight more: what its start and its parts' meeting in the CTA take.
__device__ __forceinline__ long long kv8_pieces(const Kv8AttnParams& p, const Kv8Seq& s, int from) {
  return static_cast<long long>(((s.n - 1) >> p.shift_suffix) + 1) * ((from + s.n + 31) / 32 + 8) * p.c.hkv;
}

// The line: prefix[b] = units before item b (all heads), in shared memory, filled by the whole
// CTA (THREADS threads, s_warp: KV8_SCAN_WORDS (THREADS / 32)), and its runs, PER of them a CTA
// of `grid`.  In suffix mode base[b] becomes what the prefix pass has seen to of sequence b.
constexpr int KV8_SCAN_WORDS = 3;
template <int U, int C, int THREADS, int PER>
__device__ __forceinline__ Kv8Runs kv8_line_causal(const Kv8AttnParams& p, Kv8Line& line, long long* s_warp, int grid) {
  const int tid = threadIdx.x, B = p.b.n_seqs;
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long* const prefix = line.prefix;
  long long sum = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const Kv8Seq s = kv8_seq(p.b, p.c.page_shift, b);
    // (fewer positions than new tokens: the tokens without one get zeros)
    if ((s.bad || (s.n > 0 && s.first < 0)) && blockIdx.x == 0) atomicOr(p.c.err, ERRBIT_BOUNDS);
    sum += kv8_units_seq<U, C, KV8_CAUSAL>(p, 0, s) * p.c.hkv;
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
  return Kv8Runs{total, total, static_cast<int>(min(total, static_cast<long long>(grid) * PER))};
}

// The same in the other modes.  (It runs once per launch, so its loops stay loops: see kv8_div.)
//
// Prompts with a window have tiles of much the same size, and often about as many as there are CTAs.
// Then every tile counts as long as the longest, and a CTA gets whole tiles, the same number
// each: the longest run may grow, but no tile's parts meet through the workspace, which costs
// about JOIN units of a run.  (Decode loses by it: a warp's pieces come one after the other, 1 us
// each; one sequence of 33 pieces took 12.8 us in one CTA and 10.7 in five.)
template <int U, int C, int THREADS, int PER, int JOIN, int MODE>
__device__ __forceinline__ Kv8Runs kv8_line(const Kv8AttnParams& p, Kv8Line& line, long long* s_warp, int grid) {
  line.uni = 0;
  line.shares = false;
  if constexpr (MODE == KV8_CAUSAL) return kv8_line_causal<U, C, THREADS, PER>(p, line, s_warp, grid);
  constexpr bool groups = MODE == KV8_PREFIX || MODE == KV8_SUFFIX, aligns = kv8_aligns(U, MODE);
  constexpr int W = THREADS / 32;
  static_assert(W <= 32, "a lane per warp");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = kv8_items<MODE>(p);
  const int per = (B + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  long long* const prefix = line.prefix;
  // With groups out of order or range, or a sequence that contradicts the call, nothing is shared:
  // then once more.
  bool share = groups;
#pragma unroll 1
  for (;; share = false) {
    bool fine = true;
    // the line's units; the tiles and the longest (window), or, where the passes run side by side, the
    // prefix pass's units and the suffix pass's pieces
    long long sum = 0, other = 0, pieces = 0;
    int top = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      Kv8Seq s;
      if constexpr (MODE == KV8_PREFIX) {
        s = kv8_group(p, b);
        if (!share) s.n = 0;
      } else {
        s = kv8_seq(p.b, p.c.page_shift, b);
        if constexpr (MODE == KV8_SUFFIX) line.base[b] = s.base = share ? kv8_base(p, s, b) : 0;
        if constexpr (groups) fine &= !s.bad;
        if (MODE == KV8_SUFFIX && s.n > 0) pieces += kv8_pieces(p, s, max(s.first, 0) - s.base);
      }
      // (fewer positions than new tokens: the tokens without one get zeros)
      if ((s.bad || (s.n > 0 && s.first < 0)) && blockIdx.x == 0) atomicOr(p.c.err, ERRBIT_BOUNDS);
      sum += kv8_units_seq<U, C, MODE>(p, 0, s) * p.c.hkv;
      prefix[b] = sum;                       // inside this thread's run for now
      if constexpr (aligns) {
        if (s.n > 0) {
          const int nt = ((s.n - 1) >> p.tq_shift) + 1;
          other += nt * p.c.hkv;
          top = max(top, kv8_units_tile<U, C, MODE>(p, 0, s, nt - 1));
        }
        line.base[b] = static_cast<int>(other);
      }
    }
    if constexpr (groups) {
      // (other threads than those of the items above, as long as there are enough: their loads overlap)
      const int back = THREADS - 1 - tid;
#pragma unroll 1
      for (int i = MODE == KV8_SUFFIX ? back : tid; i <= p.n_groups; i += THREADS) {
        const int b = __ldg(p.groups + i);
        fine &= b >= 0 && b <= p.b.n_seqs && (i == 0 || __ldg(p.groups + i - 1) <= b);
        if (MODE == KV8_SUFFIX && share && i < p.n_groups) {
          const Kv8Seq s = kv8_group(p, i);
          if (s.n > 0) other += static_cast<long long>(((s.n - 1) >> p.shift_prefix) + 1) * (s.len / 128 + 4) * p.c.hkv;
        }
      }
      if constexpr (MODE == KV8_PREFIX) {
#pragma unroll 1
        for (int b = back; b < p.b.n_seqs; b += THREADS) {
          const Kv8Seq s = kv8_seq(p.b, p.c.page_shift, b);
          fine &= !s.bad;
          // (the same sum as the suffix pass's, so that both divide the SMs alike)
          if (p.own && s.n > 0) pieces += kv8_pieces(p, s, max(s.first, 0) - (share ? kv8_base(p, s, b) : 0));
        }
      }
    }
    // inclusive sums over the warp's lanes, then over the warps
    long long incl = sum, rest = other;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o), x = __shfl_up_sync(0xffffffffu, rest, o);
      if (lane >= o) {
        incl += v;
        rest += x;
      }
      if constexpr (groups) pieces += __shfl_xor_sync(0xffffffffu, pieces, o);
    }
    if constexpr (aligns) top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 31) {
      s_warp[warp] = incl;
      s_warp[W + warp] = rest;
      s_warp[2 * W + warp] = aligns ? top : pieces;
    }
    const bool ok = __syncthreads_and(fine) != 0;
    long long total = lane < W ? s_warp[lane] : 0, all = lane < W ? s_warp[W + lane] : 0;
    pieces = lane < W ? s_warp[2 * W + lane] : 0;
    if constexpr (aligns) top = __reduce_max_sync(0xffffffffu, static_cast<int>(pieces));
    __syncthreads();                         // the words are read: they may be written again
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, total, o), x = __shfl_up_sync(0xffffffffu, all, o);
      if (lane >= o) {
        total += v;
        all += x;
      }
      if constexpr (groups) pieces += __shfl_xor_sync(0xffffffffu, pieces, o);
    }
    const int w1 = max(warp - 1, 0);
    const long long before = incl - sum + (warp ? __shfl_sync(0xffffffffu, total, w1) : 0);
    const long long before_rest = rest - other + (warp ? __shfl_sync(0xffffffffu, all, w1) : 0);
    total = __shfl_sync(0xffffffffu, total, 31);
    all = __shfl_sync(0xffffffffu, all, 31);
    if (groups && share && !ok) continue;
    if (groups && !ok && tid == 0 && blockIdx.x == 0) atomicOr(p.c.err, ERRBIT_BOUNDS);
    line.shares = share;
    Kv8Runs runs = {total, total, 0};
    if (groups && p.own) {
      const bool one = p.G << p.shift_prefix <= 128, rows8 = p.G << p.shift_suffix <= 8;
      const long long units = MODE == KV8_SUFFIX ? all : total;
      // (no more to the prefix pass than it has units)
      const int first = static_cast<int>(min(static_cast<long long>(grid - kv8_split(units, pieces, one, rows8, grid)), units));
      grid = MODE == KV8_SUFFIX ? grid - first : first;
    }
    runs.n = static_cast<int>(min(total, static_cast<long long>(grid) * PER));
    if constexpr (aligns) {
      static_assert(PER == 1, "a run per CTA");
      const int nt = static_cast<int>(all), waves = (nt + grid - 1) / grid;
      if (nt > 0 && static_cast<long long>(waves) * top <= kv8_div(total, grid) + JOIN) {
        line.uni = top;
        runs.n = (nt - 1) / waves + 1;
        runs.span = static_cast<long long>(runs.n) * waves * top;
        runs.total = static_cast<long long>(nt) * top;
      }
    }
    // exclusive: prefix[b] = everything before b
    long long prev = before;
    if (aligns && line.uni) prev = before_rest * line.uni;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      long long incl_b = before + prefix[b];
      if (aligns && line.uni) incl_b = (before_rest + line.base[b]) * line.uni;
      prefix[b] = prev;
      prev = incl_b;
    }
    if (tid == 0) prefix[B] = runs.total;
    __syncthreads();
    return runs;
  }
}

// Positions that the tile's last token sees.  (The tile's units are counted as if the sequence
// began at position 0 at the latest, so that with fewer positions than new tokens, first < 0, the
// last units lie past this.)
template <int MODE>
__device__ __forceinline__ int kv8_seg_end(const Kv8Seg& g, int tq_shift) {
  if constexpr (MODE == KV8_PREFIX) return g.s.len;
  return max(g.s.first + min((g.t + 1) << tq_shift, g.s.n), 0);
}

// Ends the segment that starts at unit w, x units into its tile of `all` units of the line, with
// the tile or at w_end.
template <int U, int C, int MODE>
__device__ __forceinline__ void kv8_seg_close(Kv8Seg& g, const Kv8AttnParams& p, int x, int all, long long w,
                                              long long w_end) {
  const long long left = w_end - w;
  const int end = all - x <= left ? all : x + static_cast<int>(left);
  g.x = x;
  g.len = end - x;
  g.units = all - C;
  g.u0 = max(x - C, 0);
  g.u1 = end - C;
  if constexpr (MODE == KV8_WINDOW) {
    g.low = max(g.s.first + (g.t << p.tq_shift) + 1 - p.window, 0);
    constexpr int N = kv8_granule(U);
    g.sunk = min((p.sinks + N - 1) / N, g.low / N) * N;
    g.skip = g.low / N * N - g.sunk;
    g.units = max((kv8_seg_end<MODE>(g, p.tq_shift) - g.skip + U - 1) / U, 1);
  }
  if constexpr (MODE == KV8_SUFFIX) g.units = kv8_units_tile<U, 0, MODE>(p, 0, g.s, g.t);
  if constexpr (MODE == KV8_WINDOW || kv8_aligns(U, MODE)) g.u1 = min(g.u1, g.units);
}
// The runs that hold the first and the last unit of positions of the segment's tile (the
// segment starts at unit w).
template <int U, int C, int MODE>
__device__ __forceinline__ int2 kv8_owners(const Kv8Seg& g, long long w, const Kv8Runs& runs) {
  const long long start = w - g.x;
  return make_int2(kv8_run_of<U, MODE>(runs, start + C), kv8_run_of<U, MODE>(runs, start + C + g.units - 1));
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
template <int U, int C, int MODE>
__device__ __forceinline__ Kv8Seg kv8_seg(const Kv8AttnParams& p, const Kv8Line& line, long long w, long long w_end) {
  const long long* const prefix = line.prefix;
  Kv8Seg g;
  const int lo = kv8_last_of(kv8_items<MODE>(p), [&](int i) { return prefix[i] <= w; });
  g.b = lo;
  g.s = kv8_item<MODE>(p, line.base, lo);
  long long x = w - prefix[lo];
  const long long per_head = kv8_units_seq<U, C, MODE>(p, line.uni, g.s);
  g.g = 0;
  if (p.c.hkv > 4) {
    g.g = static_cast<int>(kv8_div(x, per_head));
    x -= g.g * per_head;
  } else {
#pragma unroll 1
    for (; x >= per_head; x -= per_head) ++g.g;
  }
  const int tiles = (g.s.n + (1 << p.tq_shift) - 1) >> p.tq_shift;
  const int tl = kv8_last_of(tiles, [&](int t) { return kv8_units_before<U, C, MODE>(p, line.uni, g.s, t) <= x; });
  g.t = tl;
  const int in_tile = static_cast<int>(tl ? x - kv8_units_before<U, C, MODE>(p, line.uni, g.s, tl) : x);
  kv8_seg_close<U, C, MODE>(g, p, in_tile, kv8_units_tile<U, C, MODE>(p, line.uni, g.s, tl), w, w_end);
  return g;
}

// The segment after `g`, at unit w of the line (g was not the run's last): it begins a tile,
// the sequence's next one, or the first of the next head or sequence.
template <int U, int C, int MODE>
__device__ __forceinline__ void kv8_next(Kv8Seg& g, const Kv8AttnParams& p, const Kv8Line& line, long long w,
                                         long long w_end) {
  const long long* const prefix = line.prefix;
  const int tiles = (g.s.n + (1 << p.tq_shift) - 1) >> p.tq_shift;
  if (++g.t >= tiles) {
    g.t = 0;
    if (++g.g >= p.c.hkv) {
      g.g = 0;
      do ++g.b; while (prefix[g.b + 1] <= w);      // sequences without new tokens have no units
      g.s = kv8_item<MODE>(p, line.base, g.b);
    }
  }
  kv8_seg_close<U, C, MODE>(g, p, 0, kv8_units_tile<U, C, MODE>(p, line.uni, g.s, g.t), w, w_end);
}

}  // namespace moe
