// kv8_prompt.cu -- attention over the 8-bit key/value cache for many query rows per
// key/value head (prompts, pieces of one, more drafted tokens than the decode kernel takes),
// on tcgen05.
//
// A CTA works on one or two blocks of 128 query rows (TQ tokens x G heads each) that share
// their keys, in tiles of 128 positions; its 14 warps (128 registers each; with more than 16
// there are 96, and the scores spill) have roles:
//   warps 0-7    softmax, one query row per thread, four warps per row block
//   warps 8-11   dequantise: codes from global memory into fp16 tiles in shared memory,
//                128-byte rows with the 128-byte swizzle, two buffers each for K and V
//   warp 12      issues the MMAs
//   warp 13      plans: looks up the tiles' pages and scales ahead of the dequantising warps
// Per tile and row block, TMEM lane = query row:
//   S = Q K^T    both operands in shared memory.  fp16 holds every code exactly, and a query
//                row is scaled by a power of two to fit, so the products are exact.
//   softmax      in base 2 with the scale 2^e of the tile's values folded in, as in the decode
//                kernel: w_i = 2^(s_i + e - m), normaliser sum w_i 2^(d - e) in fp32 (m = ms + d).
//                (Dequantising brings a tile's blocks to one scale for the keys and one for the
//                values, so that no score needs a factor of its own block's.)  m moves only when a
//                row's weights pass fp16's range at either end; until then O in TMEM needs no
//                rescaling.  fp16(w) goes back to TMEM over S.
//   O += w V     w from TMEM, V from shared memory, its rows as they are (N-major operand)
// The two row blocks alternate: while one is in its softmax the tensor cores work for the
// other (order of issue: PV of block 0, next QK of block 0, PV of block 1, next QK of block 1).
// Bound: the tensor cores' 16.8 MFLOP per tile and two row blocks, 2048 cycles at the nominal
// rate (2400 at the 75 cycles that an M128 N128 K16 instruction takes in a chain), 32768
// exponentials (1024 cycles) beside them.  Measured: 2048 tokens over 31000 positions of int8,
// 16 query and 2 key/value heads of 128, in 401 us (409 with inputs that change from call to call),
// 1.25 PFLOP/s, 0.64 of the measured bf16 rate; the tensor pipe is active 56 % of the time, and what
// is left is a block's chain from scores
// through weights to the next scores, which the other block's covers only in part.  A prompt of
// 2048 tokens from the start takes 42 us: 128 tiles of 1 to 16 units each, where a tile's start
// and end (queries in, result out, some 10 thousand cycles) weigh as much as its units.
//
// With a window (MODE, see kv8_sched.cuh) a tile's places are the 16-position blocks of its sinks and of
// its windows, which the planning warp looks up one by one, so that they lie side by side; tiles
// at their edges are masked column group by column group.  2048 tokens over 14 thousand positions, a
// window of 1024 and 16 sinks, 33.4 us: 128 CTAs with a tile of 9 units each (17 us), the line and
// the first queries before them 8, the result 3.5, the join that finds nothing to do 2.  (As parts of
// an even line, sinks and window in units of 128 of their own, 54.4.)
//
// The prefix pass takes the tokens of all sequences of a group as rows of one tile and masks nothing; what
// it leaves (sums) meets each sequence's own part: with few new tokens per sequence that of the
// decode kernel, which runs beside it on the SMs that the work of either leaves it, in the
// join.  128 sequences over 32768 shared positions and 64 to 2000 of their own, e4m3, 59 us (18 at
// the tensor cores' measured rate, 76 us for a quarter of the sequences without it): 118 CTAs of
// the prefix pass 47 to 52, 34 of the other beside them, the join of 16 MB of sums 5, launches between.
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "kv8_host.h"
#include "kv8_sched.cuh"

namespace moe {

namespace {

constexpr int KP_DEQ = 4;                         // dequantising warps
constexpr int KP_THREADS = (8 + KP_DEQ + 2) * 32;
constexpr int KP_U = 128;                         // positions per tile
// A tile's start, in units.  (A shared prefix has few tiles, and the few CTAs that see the end of one and
// the start of the next have both on top of their units.  128 sequences over 32768 shared positions
// took 62.2, 62.7 and 62 us with 4, 6 and 7, 24 sequences of 4 drafts 35.2, 37.3 and 37.)
constexpr int kp_cost(int mode) { return mode == KV8_PREFIX ? 4 : 2; }
constexpr int KP_JOIN = 6;                        // parts of a tile meeting through the workspace, in units
constexpr int KP_ROWS = 128;                      // query rows per block
constexpr int KP_SLOTS = 8;                       // tiles whose scales the softmax can ask for
constexpr int KP_PLANS = 4;                       // tiles planned ahead
constexpr int KP_FEW = 4;                         // parts of a tile that a join loads at once
constexpr float KP_LOW = -7.0f;                   // 128 positions: 128 * 2^-25 = 2^-11 2^-7
// Blocks of a tile are brought to the tile's largest scale in fp16, 2^head on top of it: the
// largest code (448; for int8 the offset 1152 of its conversion) stays under fp16's largest number
// (28672 and 36864 of 65504), and a block whose scale is down to 2^-21 of the tile's largest
// keeps every bit of its codes (e4m3's smallest is 2^-9: 2^(-9 + 6 - 21) = 2^-24).
__host__ __device__ constexpr int kp_head(int fmt) { return fmt == GQA_KV8_E4M3 ? 6 : 5; }
__host__ __device__ constexpr int kp_tile(int D) { return KP_U * D * 2; }     // fp16 K or V tile (or 128 query rows)
constexpr bool kp_extra(int mode) { return mode == KV8_SUFFIX || mode == KV8_WINDOW; }        // a word per sequence
__host__ __device__ constexpr int kp_smem(int D, int B, bool extra) {
  // alignment, Q of two blocks, two K and two V tiles, scales, line, scan words, barriers and words
  return 1024 + 6 * kp_tile(D) + KP_SLOTS * 16 + 2 * KP_ROWS * 12 + (B + 2) * 8 + KP_THREADS / 32 * 3 * 8 + 25 * 8 + 64 + KP_PLANS * 128 +
         (extra ? B * 4 : 0);
}
static_assert(kp_smem(128, KV8_MAX_SEQS, true) <= 232448, "shared memory per CTA exceeds 227 KB");

// barriers: two each of the K and V buffers (full, empty) and of the row blocks, the end, and one
// per plan slot (full, empty)
enum { BAR_KF = 0, BAR_KE = 2, BAR_VF = 4, BAR_VE = 6, BAR_Q = 8, BAR_S = 10, BAR_P = 12, BAR_PV = 14, BAR_END = 16, BAR_LF = 17, BAR_LE = 21, BAR_N = 25 };

// kind::f16 with fp16 A and B, fp32 D; A K-major, B K-major or (b_mn) N-major.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// An N-major operand of 128-byte rows (64 columns of N, one row per k) with the 128-byte
// swizzle: 8-row groups 1024 bytes apart, the next 64 columns `box` bytes on.
__device__ __forceinline__ uint64_t sdesc_sw128_mn(uint32_t saddr, int box) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(box >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 bytes, a whole sector, from one thread (32-byte aligned).
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Four columns.
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// The softmax's steps that few tiles need are functions of their own: with them inside its loop a
// piece of 2048 tokens over 31000 positions took between 392 and 475 us, as the compiler's
// registers for the loop fell out, with changing inputs up to 486; now 401 and 409.  (Heads of 64
// are better off with the mask inside: 16 prompts of 512 tokens 43.6 us, 45.7 without.)
//
// What a row does not see of a tile becomes -inf: positions from `left` on, blocks of `bad`, in
// window mode those under `before` that are not under `sinks`.
__device__ __forceinline__ uint32_t kp_under(int n) { return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u; }
template <int MODE>
__device__ __forceinline__ void kp_mask(uint32_t t_s, int left, uint32_t bad, int before, int sinks) {
  uint32_t x[32];
#pragma unroll 1
  for (int c = 0; c < KP_U / 32; ++c) {
    if (MODE != KV8_WINDOW) tmem_ld32(t_s + 32 * c, x);
    uint32_t seen = kp_under(left - 32 * c);
    if (MODE == KV8_WINDOW) seen &= ~kp_under(before - 32 * c) | kp_under(sinks - 32 * c);
    if ((bad >> (2 * c)) & 1) seen &= 0xFFFF0000u;
    if ((bad >> (2 * c + 1)) & 1) seen &= 0x0000FFFFu;
    if (MODE == KV8_WINDOW) {
      // most tiles of a window have two edges, which most of their columns lie clear of
      if (__all_sync(0xffffffffu, seen == 0xFFFFFFFFu)) continue;
      tmem_ld32(t_s + 32 * c, x);
    }
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!(seen & (1u << j))) x[j] = 0xFF800000u;
    tmem_st32(t_s + 32 * c, x);
  }
  tmem_st_wait();
}
template <int MODE>
__device__ __noinline__ void kp_mask_apart(uint32_t t_s, int left, uint32_t bad, int before, int sinks) {
  kp_mask<MODE>(t_s, left, bad, before, sinks);
}
// The sum of a row's terms 2^(f x + add) of one tile.
__device__ __noinline__ float kp_bare_sum(uint32_t t_s, float f, float add) {
  float sum = 0.0f;
#pragma unroll 1
  for (int c = 0; c < KP_U; c += 4) {
    uint32_t x[4];
    tmem_ld4(t_s + c, x);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += ex2(fmaf(__uint_as_float(x[j]), f, add));
  }
  return sum;
}
// The rows whose scores lie past KV8_FAR: in the scores' place what f makes of them rounded and
// relative to `ms`.  What a row does not see stays -inf.
__device__ __noinline__ void kp_far_scores(uint32_t t_s, float f, float ms, bool far) {
#pragma unroll 1
  for (int c = 0; c < KP_U; c += 4) {
    uint32_t x[4];
    tmem_ld4(t_s + c, x);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (far && x[j] != 0xFF800000u) x[j] = __float_as_uint((kv8_end(__uint_as_float(x[j]) * f) - ms) / f);
    tmem_st4(t_s + c, x);
  }
  tmem_st_wait();
}
// The references move in the rows with `move` (m_ref and ms_ref as the softmax keeps them, ms and
// the peak in shared memory), and a tile whose weights give no terms of the normaliser adds those
// by themselves.  Returns m_ref, ms_ref, the normaliser, and what O is to be multiplied by.
__device__ __noinline__ float4 kp_refs(uint32_t t_s, float mx, float f, float e, float m_ref, float ms_ref, float l,
                                       float* s_ms, float* s_peak, bool move) {
  const float s_max = move ? kv8_end(mx * f) : KV8_NO_REF;
  const float ms = ms_ref == -INFINITY ? *s_ms : ms_ref, ms_new = fmaxf(ms, s_max);
  const float was = (ms_ref == -INFINITY ? m_ref : m_ref - ms) + (ms - ms_new);     // d in units of the new ms
  const float top = s_max - ms_new + e;
  const bool far = fabsf(ms_new) >= KV8_FAR;
  float d = was;
  if (move) d = kv8_down(top, was, KP_LOW, ms_new, *s_peak) ? top - KV8_W_FIRST : fmaxf(was, top - KV8_W_FIRST);
  *s_peak = fmaxf(*s_peak, ms_new + d);
  l *= ex2(ms - ms_new);
  m_ref = far ? d : move ? ms_new + d : m_ref;
  ms_ref = far ? -INFINITY : ms_new;
  *s_ms = ms_new;
  const bool wide = move && (d - e > KV8_SUM_TOP || far);
  if (__any_sync(0xffffffffu, wide)) {
    kp_far_scores(t_s, f, ms_new, far);
    const float sum = kp_bare_sum(t_s, f, far ? 0.0f : -ms_new);
    if (wide) l += sum;
  }
  return make_float4(m_ref, ms_ref, l, ex2(was - d));   // from no reference: 0
}
// A tile's codes, as the dequantising warps need to know them.
struct __align__(16) KpPlan {
  int rows[8];           // first code row of each 16-position block (negative: none)
  uint32_t kfac[8];      // factor of each block to the tile's scale, an fp16 pair
  uint32_t vfac[8];
  int valid;             // positions up to the tile's last token's, 0 at least; negative: no more tiles
  int pad[7];
};
static_assert(sizeof(KpPlan) == 128, "one line of shared memory");

// Two codes to fp16 times a power of two, one rounding (for int8 the offset 1152 goes with
// the multiplication: (1152 + code) f - 1152 f).
template <int FMT>
__device__ __forceinline__ uint32_t kv8_scaled_offset(uint32_t f2) {
  uint32_t r = 0;
  if constexpr (FMT == GQA_KV8_INT8) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(f2), "r"(0xE480E480u));
  return r;
}
template <int FMT>
__device__ __forceinline__ uint32_t kv8_half2_scaled(uint32_t w, int hi, uint32_t f2, uint32_t off) {
  uint32_t d;
  if constexpr (FMT == GQA_KV8_E4M3) {
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(kv8_half2<FMT>(w, hi)), "r"(f2));
  } else {
    const uint32_t x = __byte_perm(w, 0x64646464u, hi ? 0x4342 : 0x4140);
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(f2), "r"(off));
  }
  return d;
}

// A tile whose parts lie in several CTAs, left by its first CTA for the kernel that joins them.
struct __align__(16) KpTile {
  int ns;                // CTAs (0: no such tile)
  int t, g, off, n;      // tile, key/value head, the sequence's first row and new tokens
  int base;              // positions that the prefix pass has seen to
  int whole;             // prefix mode: whether the CTA has tiles of its own (set apart from the others)
  int pad;
};
constexpr int KP_SHARES = KV8_TICKET_BYTES / 4 - 1;      // prefix mode: the word of the tickets' that tells whether anything is shared
static_assert(KP_SHARES >= KV8_MAX_CTAS, "behind the tickets");

// Workspace of a part: floats of a row (O, references, normaliser), the rows of CTA c's part of
// a tile that began in CTA c_first, and the tiles to join, one entry per CTA.
__host__ __device__ constexpr int kp_ps(int D) { return kv8_row_floats(D); }
constexpr size_t KP_TILES_BYTES = KV8_MAX_CTAS * sizeof(KpTile);
__device__ __forceinline__ KpTile* kp_tiles(float* part) { return reinterpret_cast<KpTile*>(part); }
template <int D>
__device__ __forceinline__ float* kp_slot(float* part, int c, int c_first, int row) {
  static_assert(KP_TILES_BYTES % 32 == 0 && KV8_TICKET_BYTES % 32 == 0, "rows 32-byte aligned");
  return part + KP_TILES_BYTES / 4 + ((static_cast<size_t>(c) * 2 + (c == c_first)) * (2 * KP_ROWS) + row) * kp_ps(D);
}

}  // namespace

// nblk: row blocks per CTA tile (1 or 2); p.tq_shift counts the tokens of all of them.
template <int D, int FMT, int MODE>
__global__ void __launch_bounds__(KP_THREADS, 1) kv8_prompt_kernel(const __grid_constant__ Kv8AttnParams p, int nblk) {
  constexpr int TILE = kp_tile(D), KP_COST = kp_cost(MODE);
  constexpr int BOX = KP_U * 128;               // bytes of 64 dims of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* s_q = smem;
  uint8_t* s_k = smem + 2 * TILE;
  uint8_t* s_v = smem + 4 * TILE;
  // per tile {K scale, e of its V scale 2^e, nothing, blocks without a page (bits)}
  float4* s_scale = reinterpret_cast<float4*>(smem + 6 * TILE);
  KpPlan* s_plan = reinterpret_cast<KpPlan*>(s_scale + KP_SLOTS);
  float* s_rs = reinterpret_cast<float*>(s_plan + KP_PLANS);       // [256] factor of a query row's scores
  float* s_ms = s_rs + 2 * KP_ROWS;                                // [256] a row's reference, while it is far or none
  float* s_peak = s_ms + 2 * KP_ROWS;                              // [256] the highest ms + d of a row
  long long* prefix = reinterpret_cast<long long*>(s_peak + 2 * KP_ROWS);
  long long* s_warp = prefix + kv8_items<MODE>(p) + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_warp + KP_THREADS / 32 * 3);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_N);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(abort_flag) + 1);
  volatile int* s_n = reinterpret_cast<volatile int*>(s_tmem + 1);    // [2]
  volatile int* s_whole = s_n + 2;                                    // prefix mode: the run holds a whole tile
  Kv8Line line = {prefix, reinterpret_cast<int*>(s_tmem + 4), 0, false};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_KF + i), KP_DEQ);
      mbar_init(bar(BAR_KE + i), 1);
      mbar_init(bar(BAR_VF + i), KP_DEQ);
      mbar_init(bar(BAR_VE + i), 1);
      mbar_init(bar(BAR_S + i), 1);
      mbar_init(bar(BAR_P + i), 4);
      mbar_init(bar(BAR_PV + i), 1);
      mbar_init(bar(BAR_Q + i), 4);
    }
    mbar_init(bar(BAR_END), 1);
    for (int i = 0; i < KP_PLANS; ++i) {
      mbar_init(bar(BAR_LF + i), 1);
      mbar_init(bar(BAR_LE + i), KP_DEQ);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  grid_dep_wait();                              // what follows reads and writes what earlier kernels wrote
  if (MODE == KV8_PREFIX && p.own) grid_dep_launch();
  const Kv8Runs runs = kv8_line<KP_U, KP_COST, KP_THREADS, 1, KP_JOIN, MODE>(p, line, s_warp, gridDim.x);
  const int cta = blockIdx.x;
  if (MODE == KV8_PREFIX && tid == 0 && cta == 0) p.tickets[KP_SHARES] = line.shares;
  if (cta >= runs.n) {                          // the whole CTA, before any TMEM is held
    if (tid == 0) kp_tiles(p.part)[cta].ns = kp_tiles(p.part)[cta].whole = 0;
    return;
  }
  const long long w_beg = kv8_run_begin<KP_U, MODE>(runs, cta), w_end = kv8_run_begin<KP_U, MODE>(runs, cta + 1);
  const Kv8Seg first = kv8_seg<KP_U, KP_COST, MODE>(p, line, w_beg, w_end);   // where every role begins
  if (warp == 8 + KP_DEQ) {
    tmem_alloc(smem_u32(s_tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;                // S of block i at 128 i, O of block i at 256 + 128 i
  const int blk_tokens = (1 << p.tq_shift) / nblk;

  if (warp < 8) {
    // ================================================ softmax: row `r` of block `blk`
    const int blk = warp >> 2, r = tid & 127;
    if (blk < nblk) {
      const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21);    // this warp's 32 TMEM lanes
      const uint32_t t_s = t_lane + 128 * blk, t_o = t_lane + 256 + 128 * blk;
      bool dead = false;
      auto wait = [&](int b, int phase) {
        if (!dead && !__all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, p.c.err, abort_flag, p.wait_ns))) dead = true;
      };
      const uint32_t inv_g = (65535u + p.G) / p.G;       // r / G = r inv_g >> 16 for r < 128, G <= 16
      int it = 0, seg = 0;
      if (tid == 0) kp_tiles(p.part)[cta].ns = 0;        // unless a tile that begins here goes on
      if (MODE == KV8_PREFIX && tid == 0) *s_whole = 0;
      Kv8Seg sg = first;
#pragma unroll 1
      for (long long w = w_beg; w < w_end;) {
        if (w > w_beg) kv8_next<KP_U, KP_COST, MODE>(sg, p, line, w, w_end);
        w += sg.len;
        if (sg.u1 <= sg.u0) continue;      // the run ends before the tile's first positions
        const int tok0 = (sg.t << p.tq_shift) + blk * blk_tokens;
        const int tr = (r * inv_g) >> 16, tok = tok0 + tr, hh = r - tr * p.G;
        const bool live = tr < blk_tokens && tok < sg.s.n;
        // positions that the row sees; a row without a token (zeros) needs no mask
        const int see = live && MODE != KV8_PREFIX ? sg.s.first + tok + 1 : 1 << 30;
        // ---- the warp's 32 query rows, scaled into fp16, into the swizzled tile: a row per
        // D / 8 lanes, so that loads and stores are whole lines
        {
          constexpr int LPR = D / 8, RPS = 32 / LPR;             // lanes per row, rows per step
          const int qc = lane % LPR;
#pragma unroll 1
          for (int i0 = 0; i0 < 32; i0 += 8 * RPS) {
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r2 = 32 * (warp & 3) + i0 + i * RPS + lane / LPR, tb = (r2 * inv_g) >> 16;
              const int t2 = tok0 + tb;
              v[i] = make_uint4(0, 0, 0, 0);
              if (tb < blk_tokens && t2 < sg.s.n)
                v[i] = ldg_nc_v4(p.q + static_cast<size_t>(sg.s.off + t2) * p.q_stride +
                                 (sg.g * p.G + r2 - tb * p.G) * D + 8 * qc);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int r2 = 32 * (warp & 3) + i0 + i * RPS + lane / LPR;
              uint32_t* x = &v[i].x;
              uint32_t big2 = 0;
#pragma unroll
              for (int j = 0; j < 4; ++j) big2 = __vmaxu2(big2, x[j] & 0x7FFF7FFFu);
#pragma unroll
              for (int m = LPR / 2; m >= 1; m >>= 1) big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, m));
              const uint32_t big = max(big2 >> 16, big2 & 0xFFFFu);
              const int e = min(max(static_cast<int>(big >> 7) - 127 - 13, KV8_Q_MIN_EXP), KV8_Q_MAX_EXP);
              const float f = big >= 0x7F80u ? NAN : pow2i(-e);
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = pack2_f16(bf16lo(x[j]) * f, bf16hi(x[j]) * f);
              *reinterpret_cast<uint4*>(s_q + blk * TILE + (qc >> 3) * BOX + r2 * 128 + (((qc & 7) ^ (r2 & 7)) << 4)) = v[i];
              if (qc == 0) s_rs[blk * KP_ROWS + r2] = big >= 0x7F80u ? NAN : fminf(pow2i(e) * p.scale_log2, KV8_MAX_FACTOR);
            }
          }
        }
        if (tid == 0) s_n[seg & 1] = sg.u1 - sg.u0;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_Q + blk));
        const float rs = s_rs[blk * KP_ROWS + r];

        // m_ref is ms + d.  Where the scores are far, or none has been seen, it is d alone; ms lies in
        // s_ms then, and in its place minus infinity, which no tile passes by that the row sees.
        float m_ref = 0.0f, ms_ref = rs == rs ? -INFINITY : 0.0f, l = 0.0f;   // a row of NaN moves nothing
        s_ms[tid] = s_peak[tid] = KV8_NO_REF;
#pragma unroll 1
        for (int u = sg.u0; u < sg.u1; ++u, ++it) {
          wait(BAR_S + blk, it);
          if (dead) continue;
          tc_fence_after();
          const float4 sc4 = s_scale[it & (KP_SLOTS - 1)];
          const float f = fminf(fmaxf(rs * sc4.x, 1e-37f), KV8_MAX_FACTOR), e = sc4.y;  // positive: -inf stays -inf
          const uint32_t bad = __float_as_uint(sc4.w);
          // places of the unit that the row sees
          const int left = see - kv8_skip<MODE>(sg, 1 << 30) - u * KP_U;
          // window mode: those before its window, and those of the sinks
          const int before = MODE == KV8_WINDOW && live ? left - p.window : 0;
          const int sinks = MODE == KV8_WINDOW ? p.sinks - u * KP_U : 0;
          uint32_t sc[2][32];
          // A tile at the causal edge, or with a page missing: what the row does not see becomes
          // -inf in TMEM first, so that the passes below carry no mask (with it in them, the
          // compiler masked every tile: 767 us against 557).
          if (__any_sync(0xffffffffu, left < KP_U || (MODE == KV8_WINDOW && max(sinks, 0) < min(before, KP_U))) || bad) {
            if constexpr (D == 64)
              kp_mask<MODE>(t_s, left, bad, before, sinks);
            else
              kp_mask_apart<MODE>(t_s, left, bad, before, sinks);
          }
          // The scores are read twice, 32 columns at a time, the next ones while these are worked
          // on: 128 of them in registers do not fit beside the rest.  (One pass against the
          // reference of the tiles before, the weights waiting in registers until all scores are
          // seen: 518 us where two passes took 499.)
          // ---- pass 1: the maximum of s_i + e
          float mx = -INFINITY;
          tmem_ld32(t_s, sc[0]);
#pragma unroll
          for (int c = 0; c < KP_U / 32; ++c) {
            tmem_ld_wait();
            tmem_ld32(t_s + 32 * ((c + 1) % (KP_U / 32)), sc[(c + 1) & 1]);   // last: pass 2's first
            const uint32_t* x = sc[c & 1];
            float m[10];
#pragma unroll
            for (int j = 0; j < 10; ++j)
              m[j] = max3(__uint_as_float(x[3 * j]), __uint_as_float(x[3 * j + 1]), __uint_as_float(x[3 * j + 2]));
            m[0] = max3(m[0], __uint_as_float(x[30]), __uint_as_float(x[31]));
#pragma unroll
            for (int j = 0; j < 3; ++j) m[j] = max3(m[j], m[3 + j], m[6 + j]);
            mx = max3(mx, max3(m[0], m[1], m[2]), m[9]);
          }
          // ---- the references move: O and the normaliser follow
          const float w_max = fmaf(mx, f, e - m_ref);            // the largest weight's exponent
          // (a row that sees nothing here has mx = -inf, which makes the last sum NaN: it waits; moving
          // it cost runs that begin at a tile's edge 10 us of 44)
          const bool move = w_max > KV8_W_TOP || (w_max < KP_LOW && w_max > KV8_W_LOST) ||
                            fmaf(mx, 0.0f, m_ref - ms_ref - e) > KV8_SUM_TOP;
          if (__any_sync(0xffffffffu, move)) {
            tmem_ld_wait();                                      // no load is under way across the calls below
            const float4 r = kp_refs(t_s, mx, f, e, m_ref, ms_ref, l, s_ms + tid, s_peak + tid, move);
            m_ref = r.x;
            ms_ref = r.y;
            l = r.z;
            const float corr = r.w;
            tmem_ld32(t_s, sc[0]);                               // pass 2's first, again
            if (u > sg.u0) {
              wait(BAR_PV + blk, it - 1);
              if (dead) continue;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(t_o + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * corr);
                tmem_st32(t_o + 32 * c, o);
              }
            }
          }
          // ---- pass 2: weights, over the scores that were read
          {
            const float add = e - m_ref;
            const uint64_t f2 = f32x2(f, f), a2 = f32x2(add, add);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int c = 0; c < KP_U / 32; ++c) {
              tmem_ld_wait();
              if (c + 1 < KP_U / 32) tmem_ld32(t_s + 32 * (c + 1), sc[(c + 1) & 1]);
              const uint32_t* x = sc[c & 1];
              uint32_t w16[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 y = f32x2_get(fma2(f32x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), f2, a2));
                const float w0 = ex2(y.x), w1 = ex2(y.y);
                sum[j & 1] = add2(sum[j & 1], f32x2(w0, w1));
                w16[j] = pack2_f16(w0, w1);
              }
              tmem_st16(t_s + 16 * c, w16);
            }
            const float2 t = f32x2_get(add2(sum[0], sum[1]));
            const float unit = m_ref - ms_ref - e;               // of the weights, in the terms'
            if (unit <= KV8_SUM_TOP)                             // else kp_refs has added them
              l = fmaf(t.x + t.y, ex2(unit), l);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_P + blk));
        }
        // ---- the row's result
        wait(BAR_PV + blk, it - 1);
        tc_fence_after();
        const bool whole = sg.u0 == 0 && sg.u1 == sg.units;
        const float ms = ms_ref == -INFINITY ? s_ms[tid] : ms_ref;
        const float d = ms_ref == -INFINITY ? m_ref : m_ref - ms;
        float unit = ex2(d);                                     // of the weights, in the normaliser's
        const size_t at = (static_cast<size_t>(sg.s.off + tok) * p.hq + sg.g * p.G + hh);
        __nv_bfloat16* dst = live ? p.out + at * D : nullptr;
        // the row's shared positions: where the prefix pass leaves them, and where the suffix pass finds them
        float* const row = MODE == KV8_PREFIX || MODE == KV8_SUFFIX ? p.rows + at * kv8_row_floats(D) : nullptr;
        Kv8Join jn = {l, {1.0f, 0.0f}, unit};
        if (MODE == KV8_SUFFIX && sg.s.base && live) {
          jn = kv8_join(make_float4(ms, d, l, 0.0f), *reinterpret_cast<const float4*>(row + D));
          unit = jn.unit;
        }
        const float inv = jn.sum == 0.0f ? 0.0f : 1.0f / jn.sum; // a row that saw no key: zeros
        const int2 own = whole ? make_int2(cta, cta) : kv8_owners<KP_U, KP_COST, MODE>(sg, w - sg.len, runs);
        float* part = kp_slot<D>(p.part, cta, own.x, blk * KP_ROWS + r);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_o + 32 * c, o);
          tmem_ld_wait();
          if (whole && MODE == KV8_PREFIX) {
            if (live && !dead)
#pragma unroll
              for (int j = 0; j < 32; j += 8) st_global_v8(row + 32 * c + j, o + j);
          } else if (whole) {
            if (MODE == KV8_SUFFIX && sg.s.base && live)
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 v = *reinterpret_cast<const float4*>(row + 32 * c + j);
                o[j] = __float_as_uint(fmaf(jn.f[0], __uint_as_float(o[j]), jn.f[1] * v.x));
                o[j + 1] = __float_as_uint(fmaf(jn.f[0], __uint_as_float(o[j + 1]), jn.f[1] * v.y));
                o[j + 2] = __float_as_uint(fmaf(jn.f[0], __uint_as_float(o[j + 2]), jn.f[1] * v.z));
                o[j + 3] = __float_as_uint(fmaf(jn.f[0], __uint_as_float(o[j + 3]), jn.f[1] * v.w));
              }
            if (dst && !dead)
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  x[k] = jn.sum == 0.0f ? 0u
                                   : pack_bf16x2(__float_as_uint(__uint_as_float(o[j + 2 * k]) * inv * unit),
                                                 __float_as_uint(__uint_as_float(o[j + 2 * k + 1]) * inv * unit));
                if (p.out_wide) {
                  st_global_v8(dst + 32 * c + j, x);
                } else {
                  *reinterpret_cast<uint4*>(dst + 32 * c + j) = make_uint4(x[0], x[1], x[2], x[3]);
                  *reinterpret_cast<uint4*>(dst + 32 * c + j + 8) = make_uint4(x[4], x[5], x[6], x[7]);
                }
              }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8) st_global_v8(part + 32 * c + j, o + j);
          }
        }
        tc_fence_before();
        if (!whole) {
          *reinterpret_cast<float4*>(part + D) = make_float4(ms, d, l, 0.0f);
          if (tid == 0 && own.x == cta)
            kp_tiles(p.part)[cta] = KpTile{own.y - own.x + 1, sg.t, sg.g, sg.s.off, sg.s.n, sg.s.base, 0, 0};
          // (a row whose parts are joined first says so)
          if (MODE == KV8_PREFIX && own.x == cta && live) row[D + 3] = 0.0f;
        } else if (MODE == KV8_PREFIX && live) {
          *reinterpret_cast<float4*>(row + D) = make_float4(ms, d, l, dead ? 0.0f : 1.0f);
          if (tid == 0) *s_whole = 1;
        }
        ++seg;
      }
      if (tid == 0) s_n[seg & 1] = 0;      // no more segments
      if (MODE == KV8_PREFIX && tid == 0) kp_tiles(p.part)[cta].whole = *s_whole;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BAR_Q + blk));
    }
  } else if (warp < 8 + KP_DEQ) {
    // ================================================ dequantise
    constexpr int CPR = D / 16;                 // 16-byte chunks of codes per row
    constexpr int RPI = KP_DEQ * 32 / CPR;      // rows per step of the threads
    constexpr int NI = KP_U / RPI;              // steps per tile
    static_assert(RPI % 8 == 0 && KP_U % RPI == 0, "a thread's rows share their place in the swizzle");
    // 8 lanes take 4 chunks of 2 rows: what they store then lies in 8 different bank groups
    const int dt = tid - 256;
    const int cc = D == 128 ? (dt & 3) | ((dt >> 1) & 4) : dt & 3;
    const int r0 = D == 128 ? ((dt >> 2) & 1) | ((dt >> 4) << 1) : dt >> 2;
    uint8_t* const to = s_k + (cc >> 2) * BOX + r0 * 128;         // V's tiles lie 2 TILE on
    const int at0 = ((2 * (cc & 3)) ^ (r0 & 7)) << 4, at1 = ((2 * (cc & 3) + 1) ^ (r0 & 7)) << 4;
    uint4 kreg[NI], vreg[NI];
    // The codes of the tile planned in slot s.
    auto load = [&](uint4 (&reg)[NI], const uint8_t* codes, int s) {
      const int valid = s_plan[s].valid;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int row = r0 + i * RPI;
        const int at = s_plan[s].rows[row / KV8_BLOCK];
        reg[i] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && row < valid) reg[i] = ldg_nc_v4(codes + static_cast<size_t>(at + row % KV8_BLOCK) * D + 16 * cc);
      }
    };
    auto store = [&](const uint4 (&reg)[NI], uint8_t* tile, const uint32_t* fac) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const uint32_t fc = fac[(r0 + i * RPI) / KV8_BLOCK], fo = kv8_scaled_offset<FMT>(fc);
        const auto h2 = [&](uint32_t x, int hi) { return kv8_half2_scaled<FMT>(x, hi, fc, fo); };
        const uint32_t w0 = kv8_flip<FMT>(reg[i].x), w1 = kv8_flip<FMT>(reg[i].y);
        const uint32_t w2 = kv8_flip<FMT>(reg[i].z), w3 = kv8_flip<FMT>(reg[i].w);
        *reinterpret_cast<uint4*>(tile + i * RPI * 128 + at0) = make_uint4(h2(w0, 0), h2(w0, 1), h2(w1, 0), h2(w1, 1));
        *reinterpret_cast<uint4*>(tile + i * RPI * 128 + at1) = make_uint4(h2(w2, 0), h2(w2, 1), h2(w3, 0), h2(w3, 1));
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    const auto wait = [&](int b, int phase) {
      return __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, p.c.err, abort_flag, p.wait_ns)) != 0;
    };
    bool ok = wait(BAR_LF, 0) && s_plan[0].valid >= 0;
    if (ok) {
      load(kreg, p.c.codes[0], 0);
      load(vreg, p.c.codes[1], 0);
    }
#pragma unroll 1
    for (int it = 0; ok; ++it) {
      const int s = it & 1, ph = (it >> 1) & 1, slot = it & (KP_PLANS - 1), next = (it + 1) & (KP_PLANS - 1);
      if (!wait(BAR_KE + s, ph ^ 1)) break;
      store(kreg, to + s * TILE, s_plan[slot].kfac);
      if (lane == 0) mbar_arrive(bar(BAR_KF + s));
      if (!wait(BAR_LF + next, (it + 1) / KP_PLANS)) break;
      ok = s_plan[next].valid >= 0;
      if (ok) load(kreg, p.c.codes[0], next);
      if (!wait(BAR_VE + s, ph ^ 1)) break;
      store(vreg, to + (2 + s) * TILE, s_plan[slot].vfac);
      if (lane == 0) {
        mbar_arrive(bar(BAR_VF + s));
        mbar_arrive(bar(BAR_LE + slot));
      }
      if (ok) load(vreg, p.c.codes[1], next);
    }
  } else {
    if (warp == 9 + KP_DEQ) {
      // ================================================ plan: the tiles' pages and scales
      // Lanes 0-7 look after the tile's 8 K blocks, lanes 8-15 after its V blocks.  The
      // dequantising warps are left with loads, conversions and stores, whose instructions are
      // what the softmax competes with (8900 warp instructions a tile in all: 499 us; 7150: 390).
      const int lb = lane & 7;
      Kv8Seg sg = first;
      bool ok = true;
      int it = 0;
#pragma unroll 1
      for (long long w = w_beg; ok; w += sg.len) {
        if (w > w_beg && w < w_end) kv8_next<KP_U, KP_COST, MODE>(sg, p, line, w, w_end);
        const bool more = w < w_end;
        const int end = kv8_seg_end<MODE>(sg, p.tq_shift);
        const int* table = kv8_table<MODE>(p, sg.b);
        int u = more ? sg.u0 : 0;
        const int u1 = more ? sg.u1 : 1;               // at the end one more plan: no more tiles
        int pid = -1;
        const auto place = [&](int u) {                // where the lane's block of unit u begins
          const int i = u * KP_U + lb * KV8_BLOCK;
          return i + kv8_skip<MODE>(sg, i);
        };
        const auto look = [&] {
          const int pos = place(u);
          pid = more && u < u1 && pos < end ? __ldg(table + (pos >> p.c.page_shift)) : -1;
        };
        look();
#pragma unroll 1
        while (u < u1) {
          const int pos = place(u);
          const bool exists = more && pos < end, bad = exists && (pid < 0 || pid >= p.c.n_pages);
          int row = -1;
          float scale = 0.0f;
          if (exists && !bad) {
            row = ((pid * p.c.hkv + sg.g) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1));   // below 2^31
            scale = __ldg(p.c.scales[(lane >> 3) & 1] + row / KV8_BLOCK);
          }
          // A sequence with fewer positions than new tokens has units past its end: nothing valid
          // in them, which is not the mark of the end.
          const int valid = more ? max(end - kv8_skip<MODE>(sg, 1 << 30) - u * KP_U, 0) : -1;
          ++u;
          look();                                      // the next tile's pages meanwhile
          const uint32_t bads = __ballot_sync(0xffffffffu, bad) & 0xFFu;
          if (bads && lane == 0) atomicOr(p.c.err, ERRBIT_BOUNDS);
          constexpr int HEAD = kp_head(FMT);
          const int e = row >= 0 ? max(scale_exp(fmaxf(scale, 0.0f)), KV8_MIN_EXP) : KV8_MIN_EXP;
          int t = e;                                   // the largest of the 8 blocks
#pragma unroll
          for (int m = 4; m >= 1; m >>= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, m));
          const float f = pow2i(max(e - t + HEAD, -126));
          const int kt = __shfl_sync(0xffffffffu, t, 0), vt = __shfl_sync(0xffffffffu, t, 8);
          const int slot = it & (KP_PLANS - 1);
          ok = __all_sync(0xffffffffu, mbar_wait(bar(BAR_LE + slot), ((it / KP_PLANS) & 1) ^ 1, p.c.err, abort_flag, p.wait_ns));
          if (!ok) break;
          KpPlan* plan = s_plan + slot;
          if (lane < 8) {
            plan->rows[lane] = row;
            plan->kfac[lane] = pack2_f16(f, f);
          } else if (lane < 16) {
            plan->vfac[lane - 8] = pack2_f16(f, f);
          } else if (lane == 16) {
            plan->valid = valid;
            s_scale[it & (KP_SLOTS - 1)] =
                make_float4(pow2i(kt - HEAD), static_cast<float>(vt - HEAD), 0.0f, __uint_as_float(bads));
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(BAR_LF + slot));
          ++it;
        }
        if (!more) break;
      }
    } else if (warp == 8 + KP_DEQ) {
      // ================================================ MMA issue
      // The whole warp follows the loop and one elected lane issues, with the row block and the
      // buffer known at compile time, so that every descriptor is a uniform base plus a constant.
      // (A lane with a loop of its own issued an MMA every 120 cycles: 570 us where this took
      // 470.  A warp per row block let the blocks fall into step, both in their softmax and then
      // both on the tensor cores: 560 us.)
      constexpr uint32_t ID_S = idesc_f16(KP_ROWS, KP_U, 0), ID_O = idesc_f16(KP_ROWS, D, 1);
      const bool leader = elect_one();
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint64_t d_q = sdesc_sw128(smem_u32(s_q)), d_k = sdesc_sw128(smem_u32(s_k));
      const uint64_t d_v = sdesc_sw128_mn(smem_u32(s_v), BOX);
      using Zero = std::integral_constant<int, 0>;
      using One = std::integral_constant<int, 1>;
      auto qk = [&](auto block, auto buffer) {    // descriptors advance in units of 16 bytes
        constexpr int i = decltype(block)::value, s = decltype(buffer)::value;
        if (leader) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int at = (k >> 2) * (BOX >> 4) + 2 * (k & 3);
            umma_bf16(tm + 128 * i, d_q + (i * (TILE >> 4) + at), d_k + (s * (TILE >> 4) + at), ID_S, k > 0);
          }
          umma_commit(bar(BAR_S + i));
          if (i == nblk - 1) umma_commit(bar(BAR_KE + s));
        }
        __syncwarp();
      };
      auto pv = [&](auto block, auto buffer, uint32_t acc) {
        constexpr int i = decltype(block)::value, s = decltype(buffer)::value;
        if (leader) {
#pragma unroll
          for (int k = 0; k < KP_U / 16; ++k)
            umma_f16_ts(tm + 256 + 128 * i, tm + 128 * i + 8 * k, d_v + (s * (TILE >> 4) + k * (2048 >> 4)), ID_O,
                        k > 0 ? 1u : acc);
          umma_commit(bar(BAR_PV + i));
          if (i == nblk - 1) umma_commit(bar(BAR_VE + s));
        }
        __syncwarp();
      };
      auto wait = [&](int b, int phase) {
        const bool ok = __all_sync(0xffffffffu, mbar_wait(bar(b), phase & 1, p.c.err, abort_flag, p.wait_ns));
        tc_fence_after();
        return ok;
      };
      int it = 0;
      // tile `it`, in buffer S: PV of each block, then QK of its next tile
      auto step = [&](auto buffer, bool begun, bool next) {
        constexpr int s = decltype(buffer)::value;
        using Other = std::integral_constant<int, 1 - s>;
        // a poll takes 300 cycles even when nothing is left to wait for: the buffers' come first
        if (!wait(BAR_VF + s, it >> 1) || (next && !wait(BAR_KF + 1 - s, (it + 1) >> 1)) || !wait(BAR_P, it)) return false;
        pv(Zero{}, buffer, begun);
        if (next) qk(Zero{}, Other{});
        if (nblk == 2) {
          if (!wait(BAR_P + 1, it)) return false;
          pv(One{}, buffer, begun);
          if (next) qk(One{}, Other{});
        }
        return true;
      };
      bool ok = true;
#pragma unroll 1
      for (int seg = 0; ok; ++seg) {
        ok = wait(BAR_Q, seg);
        if (!ok) break;
        const int n = s_n[seg & 1];               // the segment's tiles, told by the softmax (0: no more)
        if (n == 0) break;
        ok = wait(BAR_KF + (it & 1), it >> 1) && (nblk == 1 || wait(BAR_Q + 1, seg));
        if (!ok) break;
        if (it & 1) {
          qk(Zero{}, One{});
          if (nblk == 2) qk(One{}, One{});
        } else {
          qk(Zero{}, Zero{});
          if (nblk == 2) qk(One{}, Zero{});
        }
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j, ++it) ok = it & 1 ? step(One{}, j > 0, j + 1 < n) : step(Zero{}, j > 0, j + 1 < n);
      }
      // every MMA issued has to land before the memory goes away
      if (leader) umma_commit(bar(BAR_END));
      __syncwarp();
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(bar(BAR_END), 0) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 8 + KP_DEQ) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the tiles that lie in several CTAs: a block per tile (by its first CTA)
// and 8 rows, a warp per row, the parts in the order of the line.  (The last CTA of a tile
// joining them itself took over 60 us of a 150 us prompt: 256 rows by one CTA's 8 warps.)
template <int D>
__global__ void __launch_bounds__(256) kv8_prompt_join_kernel(const __grid_constant__ Kv8AttnParams p, int nblk) {
  grid_dep_wait();
  const int c0 = blockIdx.x, lane = threadIdx.x & 31;
  const KpTile tl = kp_tiles(p.part)[c0];
  if (tl.ns == 0) return;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int blk_tokens = (1 << p.tq_shift) / nblk, r = row & (KP_ROWS - 1), tb = r / p.G;
  const int tok = (tl.t << p.tq_shift) + row / KP_ROWS * blk_tokens + tb;
  if (tb >= blk_tokens || tok >= tl.n) return;
  constexpr int PL = D / 32;                    // dims per lane
  const auto slot = [&](int i) { return kp_slot<D>(p.part, c0 + i, c0, row); };
  float M = KV8_NO_REF, top = -INFINITY, L = 0.0f, O[PL];           // references ms and d of the whole
#pragma unroll
  for (int k = 0; k < PL; ++k) O[k] = 0.0f;
  const auto fetch = [&](int i, float (&v)[PL]) {
    const float* src = slot(i) + PL * lane;
    if constexpr (PL == 4)
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
    else
      *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(src);
  };
  if (tl.ns <= KP_FEW) {
    // few parts (tiles of a long prompt): all loads at once
    float ml[KP_FEW], dl[KP_FEW], ll[KP_FEW];
    float v[KP_FEW][PL];
#pragma unroll
    for (int i = 0; i < KP_FEW; ++i) {
      ml[i] = KV8_NO_REF;
      dl[i] = -INFINITY;
      if (i < tl.ns) {
        const float4 r = *reinterpret_cast<const float4*>(slot(i) + D);
        ml[i] = r.x;
        dl[i] = r.y;
        ll[i] = r.z;
        fetch(i, v[i]);
      }
      M = fmaxf(M, ml[i]);
    }
#pragma unroll
    for (int i = 0; i < KP_FEW; ++i) top = fmaxf(top, ml[i] - M + dl[i]);
#pragma unroll
    for (int i = 0; i < KP_FEW; ++i) {
      if (i >= tl.ns) break;
      const float f = ex2(ml[i] - M + dl[i] - top);
      L = fmaf(ex2(ml[i] - M), ll[i], L);
#pragma unroll
      for (int k = 0; k < PL; ++k) O[k] = fmaf(f, v[i][k], O[k]);
    }
  } else {
    // many (few query rows over a long cache): lane i keeps the weights of parts i, i + 32, ...
    constexpr int PER = (KV8_MAX_CTAS + 31) / 32;
    float wt[PER], ml[PER], ll[PER];              // wt: d until it is the weight
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = lane + 32 * k;
      ml[k] = KV8_NO_REF;
      wt[k] = -INFINITY;
      ll[k] = 0.0f;
      if (i < tl.ns) {
        const float4 r = *reinterpret_cast<const float4*>(slot(i) + D);
        ml[k] = r.x;
        wt[k] = r.y;
        ll[k] = r.z;
      }
      M = fmaxf(M, ml[k]);
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      L = fmaf(ex2(ml[k] - M), ll[k], L);
      wt[k] += ml[k] - M;
      top = fmaxf(top, wt[k]);
    }
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
#pragma unroll
    for (int k = 0; k < PER; ++k) wt[k] = ex2(wt[k] - top);
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int n = min(tl.ns - 32 * k, 32);
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const float f = __shfl_sync(0xffffffffu, wt[k], i);
        float v[PL];
        fetch(32 * k + i, v);
#pragma unroll
        for (int j = 0; j < PL; ++j) O[j] = fmaf(f, v[j], O[j]);
      }
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;   // a row that saw no key: zeros
  const float unit = ex2(top);
  __nv_bfloat16* dst = p.out + (static_cast<size_t>(tl.off + tok) * p.hq + tl.g * p.G + r - tb * p.G) * D + PL * lane;
#pragma unroll
  for (int k = 0; k < PL; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) =
        pack_bf16x2(__float_as_uint(O[k] * inv * unit), __float_as_uint(O[k + 1] * inv * unit));
}

// The same for the other modes, whose tiles are few or have many parts.  Every block makes the list of
// tiles to join, as chunks of work of the same size, and takes its share of them, so no block is
// launched for a tile that is not there (4864 of them cost 6 us).  A row's parts are divided among 1, 2, 4
// or 8 warps, each of which has its loads under way together, and the warps' sums meet in shared
// memory in order.  In prefix mode the result stays in sums, for the suffix pass to take up; or, where
// that pass ran beside it, meets that pass's sums, as those of rows do whose tile was whole.
constexpr int KJ_WARPS = 8, KJ_PER_SM = 4;  // and blocks of a launch per SM
constexpr int KJ_FLIGHT = 6;                // parts of a warp whose loads are under way together
__device__ __forceinline__ int kj_split(int ns, int most) {          // warps of a row, a lane per part at least
  const int wish = ns <= KJ_FLIGHT ? 1 : ns <= 2 * KJ_FLIGHT ? 2 : ns <= 4 * KJ_FLIGHT ? 4 : 8;
  return max(min(wish, most), ns <= 32 ? 1 : ns <= 64 ? 2 : ns <= 128 ? 4 : 8);
}
template <int D, int MODE>
__global__ void __launch_bounds__(KJ_WARPS * 32, KJ_PER_SM) kv8_parts_join_kernel(const __grid_constant__ Kv8AttnParams p, int nblk, int ctas, int most) {
  constexpr int PL = D / 32;                    // dims per lane
  __shared__ int s_start[KV8_MAX_CTAS + 1], s_sum[KJ_WARPS];
  __shared__ KpTile s_tile[KV8_MAX_CTAS];
  __shared__ float s_o[KJ_WARPS][D];
  __shared__ float4 s_ref[KJ_WARPS];
  static_assert(KV8_MAX_CTAS <= KJ_WARPS * 32, "a thread per tile");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tq = 1 << p.tq_shift, blk_tokens = tq / nblk;
  const auto rows_of = [&](const KpTile& t) { return min(tq, t.n - (t.t << p.tq_shift)) * p.G; };
  grid_dep_wait();
  const bool both = MODE == KV8_PREFIX && p.own;         // the two passes ran side by side
  int chunks = 0, whole = 0;
  if (tid < ctas && !(both && !p.tickets[KP_SHARES])) {
    const KpTile t = kp_tiles(p.part)[tid];
    s_tile[tid] = t;
    whole = t.whole;
    if (t.ns > 0) chunks = (rows_of(t) * kj_split(t.ns, most) + KJ_WARPS - 1) / KJ_WARPS;
  }
  int incl = chunks;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < KJ_WARPS; ++w) {
    if (w < warp) incl += s_sum[w];
    total += s_sum[w];
  }
  if (tid < KV8_MAX_CTAS) s_start[tid] = incl - chunks;
  whole = __syncthreads_or(whole);
  // a row's two sums, meeting: that of its shared positions (m, d, l, O) and its own
  float4 own = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float own_o[PL];
  const auto fetch_own = [&](size_t at) {        // (on its way while the shared sums are)
    const float* src = p.own + at * kv8_row_floats(D);
    own = *reinterpret_cast<const float4*>(src + D);
#pragma unroll
    for (int q = 0; q < PL; q += 2) *reinterpret_cast<float2*>(own_o + q) = *reinterpret_cast<const float2*>(src + PL * lane + q);
  };
  const auto meet = [&](size_t at, const float4& shared, float (&O)[PL]) {
    if (own.w == 0.0f) return;                   // the sequence did without the prefix pass
    const Kv8Join jn = kv8_join(own, shared);
    const float inv = jn.sum == 0.0f ? 0.0f : 1.0f / jn.sum;
    __nv_bfloat16* dst = p.out + at * D + PL * lane;
#pragma unroll
    for (int q = 0; q < PL; q += 2)
      *reinterpret_cast<uint32_t*>(dst + q) =
          pack_bf16x2(__float_as_uint(fmaf(jn.f[0], own_o[q], jn.f[1] * O[q]) * inv * jn.unit),
                      __float_as_uint(fmaf(jn.f[0], own_o[q + 1], jn.f[1] * O[q + 1]) * inv * jn.unit));
  };
  const int off0 = both && whole ? __ldg(p.b.offsets) : 0;
  const int rows = both && whole ? (__ldg(p.b.offsets + p.b.n_seqs) - off0) * p.hq : 0;
#pragma unroll 1
  for (int item = blockIdx.x; item < total + (rows + KJ_WARPS - 1) / KJ_WARPS; item += gridDim.x) {
    if (item >= total) {
      // a row of the batch, if its tile was whole
      const int i = (item - total) * KJ_WARPS + warp;
      if (i >= rows) continue;
      const size_t at = static_cast<size_t>(off0) * p.hq + i;
      fetch_own(at);
      const float* src = p.rows + at * kv8_row_floats(D);
      const float4 ref = *reinterpret_cast<const float4*>(src + D);
      if (ref.w == 0.0f) continue;
      float O[PL];
#pragma unroll
      for (int q = 0; q < PL; ++q) O[q] = src[PL * lane + q];
      meet(at, ref, O);
      continue;
    }
    const int c0 = kv8_last_of(ctas, [&](int i) { return s_start[i] <= item; });
    const KpTile tl = s_tile[c0];
    const int S = kj_split(tl.ns, most), sub = warp & (S - 1);
    const int j = ((item - s_start[c0]) * KJ_WARPS + warp) / S;         // the row among the tile's
    const bool live = j < rows_of(tl);
    const int tok = j / p.G, hh = j - tok * p.G, blk = tok >= blk_tokens;
    const int row = blk * KP_ROWS + (tok - blk * blk_tokens) * p.G + hh;
    const auto slot = [&](int i) { return kp_slot<D>(p.part, c0 + i, c0, row); };
    float m = KV8_NO_REF, d = -INFINITY, l = 0.0f, v[KJ_FLIGHT][PL];
    const int i = sub + lane * S;                                       // this lane's part
    const int n = live ? (tl.ns - sub + S - 1) / S : 0;                 // the warp's parts, at most 32
    const auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < KJ_FLIGHT; ++k)
        if (k0 + k < n) {
          const float* src = slot(sub + (k0 + k) * S) + PL * lane;
          if constexpr (PL == 4)
            *reinterpret_cast<float4*>(v[k]) = *reinterpret_cast<const float4*>(src);
          else
            *reinterpret_cast<float2*>(v[k]) = *reinterpret_cast<const float2*>(src);
        }
    };
    if (lane < n) {
      const float4 r = *reinterpret_cast<const float4*>(slot(i) + D);
      m = r.x;
      d = r.y;
      l = r.z;
    }
    fetch(0);
    const size_t at = static_cast<size_t>(tl.off + (tl.t << p.tq_shift) + tok) * p.hq + tl.g * p.G + hh;
    if (both && sub == 0 && live) fetch_own(at);
    float M = m;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = ex2(m - M) * l;
    d += m - M;
    float top = d;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      L += __shfl_xor_sync(0xffffffffu, L, o);
    }
    const float wt = ex2(d - top);
    float O[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) O[k] = 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += KJ_FLIGHT) {
      if (k0) fetch(k0);
#pragma unroll
      for (int k = 0; k < KJ_FLIGHT; ++k) {
        const float f = __shfl_sync(0xffffffffu, wt, (k0 + k) & 31);
        if (k0 + k < n)
#pragma unroll
          for (int q = 0; q < PL; ++q) O[q] = fmaf(f, v[k][q], O[q]);
      }
    }
    if (S > 1) {
#pragma unroll
      for (int q = 0; q < PL; ++q) s_o[warp][PL * lane + q] = O[q];
      if (lane == 0) s_ref[warp] = make_float4(M, top, L, 0.0f);
      __syncthreads();
      if (sub == 0) {
#pragma unroll 1
        for (int w = warp + 1; w < warp + S; ++w) {
          const float4 a = make_float4(M, top, L, 0.0f), b = s_ref[w];
          const Kv8Join jn = kv8_join(a, b);
          top = fmaxf(a.x - fmaxf(a.x, b.x) + a.y, b.x - fmaxf(a.x, b.x) + b.y);
          M = fmaxf(a.x, b.x);
          L = jn.sum;
#pragma unroll
          for (int q = 0; q < PL; ++q) O[q] = fmaf(jn.f[0], O[q], jn.f[1] * s_o[w][PL * lane + q]);
        }
      }
      __syncthreads();
    }
    if (sub != 0 || !live) continue;
    if (both) {
      meet(at, make_float4(M, top, L, 0.0f), O);
      continue;
    }
    if constexpr (MODE == KV8_PREFIX) {
      float* to = p.rows + at * kv8_row_floats(D);
#pragma unroll
      for (int q = 0; q < PL; ++q) to[PL * lane + q] = O[q];
      if (lane == 0) *reinterpret_cast<float4*>(to + D) = make_float4(M, top, L, 0.0f);
      continue;
    }
    float unit = ex2(top);
    if (MODE == KV8_SUFFIX && tl.base) {           // the row's shared positions
      const float* src = p.rows + at * kv8_row_floats(D);
      const Kv8Join jn = kv8_join(make_float4(M, top, L, 0.0f), *reinterpret_cast<const float4*>(src + D));
#pragma unroll
      for (int q = 0; q < PL; ++q) O[q] = fmaf(jn.f[0], O[q], jn.f[1] * src[PL * lane + q]);
      L = jn.sum;
      unit = jn.unit;
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L; // a row that saw no key: zeros
    __nv_bfloat16* dst = p.out + at * D + PL * lane;
#pragma unroll
    for (int q = 0; q < PL; q += 2)
      *reinterpret_cast<uint32_t*>(dst + q) =
          pack_bf16x2(__float_as_uint(O[q] * inv * unit), __float_as_uint(O[q + 1] * inv * unit));
  }
}

// ---------------------------------------------------------------- host side
size_t kv8_prompt_ws_bytes(int D) {
  return KV8_TICKET_BYTES + KP_TILES_BYTES +
         static_cast<size_t>(KV8_MAX_CTAS) * 2 * (2 * KP_ROWS) * kp_ps(D) * sizeof(float);
}

namespace {
template <int D, int FMT, int MODE>
cudaError_t launch_prompt(const Kv8AttnParams& p, int nblk, int grid, int dev, cudaStream_t s) {
  static bool set[KV8_MAX_DEVICES] = {};
  auto* k = kv8_prompt_kernel<D, FMT, MODE>;
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kp_smem(D, KV8_MAX_SEQS, kp_extra(MODE)));
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const cudaError_t e = launch_pdl(k, dim3(grid), dim3(KP_THREADS),
                                   kp_smem(D, MODE == KV8_PREFIX ? p.n_groups : p.b.n_seqs, kp_extra(MODE)), s, p, nblk);
  if (e != cudaSuccess) return e;
  if constexpr (MODE == KV8_CAUSAL)
    return launch_pdl(kv8_prompt_join_kernel<D>, dim3(grid, nblk * KP_ROWS / 8), dim3(256), 0, s, p, nblk);
  return cudaSuccess;
}
// Tokens of a row block: the largest power of two whose rows fit.
int kp_block_shift(int G) {
  int shift = 0;
  while ((2 << shift) * G <= KP_ROWS) ++shift;
  return shift;
}
}  // namespace

int kv8_prompt_shift(int G, int tokens) {
  const int shift = kp_block_shift(G);
  return shift + (tokens > (1 << shift));
}
int kv8_prompt_tokens(const Kv8AttnParams& p, int mode) {
  return mode == KV8_PREFIX ? (p.b.n_tokens - 1) / p.n_groups + 1 : p.b.max_new;
}

template <int MODE>
cudaError_t launch_kv8_join(Kv8AttnParams p, int D, int grid, cudaStream_t s) {
  p.tq_shift = kv8_prompt_shift(p.G, kv8_prompt_tokens(p, MODE));
  const int nblk = 1 + p.tq_shift - kp_block_shift(p.G);
  // warps of a row: no more than leave every row a place in one round of the blocks (2048 rows of 15
  // parts: 7 us with 4 warps in two rounds, 5 with 2 in one)
  int most = 1;
  while (most < KJ_WARPS && 2ll * most * p.b.n_tokens * p.hq <= 1ll * grid * KJ_PER_SM * KJ_WARPS) most *= 2;
  return launch_pdl(D == 128 ? kv8_parts_join_kernel<128, MODE> : kv8_parts_join_kernel<64, MODE>, dim3(grid * KJ_PER_SM),
                    dim3(KJ_WARPS * 32), 0, s, p, nblk, grid, most);
}

template <int MODE>
cudaError_t launch_kv8_prompt(Kv8AttnParams p, int D, int format, int grid, int dev, cudaStream_t s) {
  p.tq_shift = kv8_prompt_shift(p.G, kv8_prompt_tokens(p, MODE));
  const int nblk = 1 + p.tq_shift - kp_block_shift(p.G);
  if (MODE == KV8_WINDOW) p.win_units = kv8_win_units(KP_U, 1 << p.tq_shift, p.window, p.sinks);
  const bool e4 = format == GQA_KV8_E4M3;
  cudaError_t e;
  if (D == 128)
    e = e4 ? launch_prompt<128, GQA_KV8_E4M3, MODE>(p, nblk, grid, dev, s)
           : launch_prompt<128, GQA_KV8_INT8, MODE>(p, nblk, grid, dev, s);
  else
    e = e4 ? launch_prompt<64, GQA_KV8_E4M3, MODE>(p, nblk, grid, dev, s)
           : launch_prompt<64, GQA_KV8_INT8, MODE>(p, nblk, grid, dev, s);
  if constexpr (MODE == KV8_WINDOW || MODE == KV8_SUFFIX)
    if (e == cudaSuccess) e = launch_kv8_join<MODE>(p, D, grid, s);
  return e;
}
template cudaError_t launch_kv8_join<KV8_PREFIX>(Kv8AttnParams, int, int, cudaStream_t);
template cudaError_t launch_kv8_prompt<KV8_CAUSAL>(Kv8AttnParams, int, int, int, int, cudaStream_t);
template cudaError_t launch_kv8_prompt<KV8_WINDOW>(Kv8AttnParams, int, int, int, int, cudaStream_t);
template cudaError_t launch_kv8_prompt<KV8_PREFIX>(Kv8AttnParams, int, int, int, int, cudaStream_t);
template cudaError_t launch_kv8_prompt<KV8_SUFFIX>(Kv8AttnParams, int, int, int, int, cudaStream_t);

}  // namespace moe
