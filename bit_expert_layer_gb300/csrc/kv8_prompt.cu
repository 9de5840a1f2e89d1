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
constexpr int KP_COST = 2;                        // a tile's start, in units
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
__host__ __device__ constexpr int kp_smem(int D, int B) {
  // alignment, Q of two blocks, two K and two V tiles, scales, line, scan words, barriers and words
  return 1024 + 6 * kp_tile(D) + KP_SLOTS * 16 + 2 * KP_ROWS * 12 + (B + 2) * 8 + KP_THREADS / 32 * 8 + 25 * 8 + 64 + KP_PLANS * 128;
}
static_assert(kp_smem(128, KV8_MAX_SEQS) <= 232448, "shared memory per CTA exceeds 227 KB");

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
// Two fp32 fused multiply-adds / additions in one instruction.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 f32x2_get(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The softmax's steps that few tiles need are functions of their own: with them inside its loop a
// piece of 2048 tokens over 31000 positions took between 392 and 475 us, as the compiler's
// registers for the loop fell out, with changing inputs up to 486; now 401 and 409.  (Heads of 64
// are better off with the mask inside: 16 prompts of 512 tokens 43.6 us, 45.7 without.)
//
// What a row does not see of a tile becomes -inf: positions from `left` on, blocks of `bad`.
__device__ __forceinline__ void kp_mask(uint32_t t_s, int left, uint32_t bad) {
  uint32_t x[32];
#pragma unroll 1
  for (int c = 0; c < KP_U / 32; ++c) {
    tmem_ld32(t_s + 32 * c, x);
    const int n = left - 32 * c;
    uint32_t seen = n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
    if ((bad >> (2 * c)) & 1) seen &= 0xFFFF0000u;
    if ((bad >> (2 * c + 1)) & 1) seen &= 0x0000FFFFu;
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!(seen & (1u << j))) x[j] = 0xFF800000u;
    tmem_st32(t_s + 32 * c, x);
  }
  tmem_st_wait();
}
__device__ __noinline__ void kp_mask_apart(uint32_t t_s, int left, uint32_t bad) { kp_mask(t_s, left, bad); }
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
  int pad[3];
};

// Workspace of a part: floats of a row (O, references, normaliser), the rows of CTA c's part of
// a tile that began in CTA c_first, and the tiles to join, one entry per CTA.
__host__ __device__ constexpr int kp_ps(int D) { return D + 8; }      // 32-byte rows
constexpr size_t KP_TILES_BYTES = KV8_MAX_CTAS * sizeof(KpTile);
__device__ __forceinline__ KpTile* kp_tiles(float* part) { return reinterpret_cast<KpTile*>(part); }
template <int D>
__device__ __forceinline__ float* kp_slot(float* part, int c, int c_first, int row) {
  static_assert(KP_TILES_BYTES % 32 == 0 && KV8_TICKET_BYTES % 32 == 0, "rows 32-byte aligned");
  return part + KP_TILES_BYTES / 4 + ((static_cast<size_t>(c) * 2 + (c == c_first)) * (2 * KP_ROWS) + row) * kp_ps(D);
}

}  // namespace

// nblk: row blocks per CTA tile (1 or 2); p.tq_shift counts the tokens of all of them.
template <int D, int FMT>
__global__ void __launch_bounds__(KP_THREADS, 1) kv8_prompt_kernel(const __grid_constant__ Kv8AttnParams p, int nblk) {
  constexpr int TILE = kp_tile(D);
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
  long long* s_warp = prefix + p.b.n_seqs + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_warp + KP_THREADS / 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_N);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(abort_flag) + 1);
  volatile int* s_n = reinterpret_cast<volatile int*>(s_tmem + 1);    // [2]
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
  Kv8Runs runs;
  runs.total = kv8_line<KP_U, KP_COST, KP_THREADS>(p, prefix, s_warp);
  runs.n = static_cast<int>(min(runs.total, static_cast<long long>(gridDim.x)));
  const int cta = blockIdx.x;
  if (cta >= runs.n) {                          // the whole CTA, before any TMEM is held
    if (tid == 0) kp_tiles(p.part)[cta].ns = 0;
    return;
  }
  const long long w_beg = kv8_run_begin(runs, cta), w_end = kv8_run_begin(runs, cta + 1);
  const Kv8Seg first = kv8_seg<KP_U, KP_COST>(p, prefix, w_beg, w_end);   // where every role begins
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
      Kv8Seg sg = first;
#pragma unroll 1
      for (long long w = w_beg; w < w_end;) {
        if (w > w_beg) kv8_next<KP_U, KP_COST>(sg, p, prefix, w, w_end);
        w += sg.len;
        if (sg.u1 <= sg.u0) continue;      // the run ends before the tile's first positions
        const int tok0 = (sg.t << p.tq_shift) + blk * blk_tokens;
        const int tr = (r * inv_g) >> 16, tok = tok0 + tr, hh = r - tr * p.G;
        const bool live = tr < blk_tokens && tok < sg.s.n;
        // positions that the row sees; a row without a token (zeros) needs no mask
        const int see = live ? sg.s.first + tok + 1 : 1 << 30;
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
          const int left = see - u * KP_U;                       // positions of the tile that the row sees
          uint32_t sc[2][32];
          // A tile at the causal edge, or with a page missing: what the row does not see becomes
          // -inf in TMEM first, so that the passes below carry no mask (with it in them, the
          // compiler masked every tile: 767 us against 557).
          if (__any_sync(0xffffffffu, left < KP_U) || bad) {
            if constexpr (D == 64)
              kp_mask(t_s, left, bad);
            else
              kp_mask_apart(t_s, left, bad);
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
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;           // a row that saw no key: zeros
        const float ms = ms_ref == -INFINITY ? s_ms[tid] : ms_ref;
        const float d = ms_ref == -INFINITY ? m_ref : m_ref - ms;
        const float unit = ex2(d);                               // of the weights, in the normaliser's
        __nv_bfloat16* dst =
            live ? p.out + (static_cast<size_t>(sg.s.off + tok) * p.hq + sg.g * p.G + hh) * D : nullptr;
        const int2 own = whole ? make_int2(cta, cta) : kv8_owners<KP_COST>(sg, w - sg.len, runs);
        float* part = kp_slot<D>(p.part, cta, own.x, blk * KP_ROWS + r);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_o + 32 * c, o);
          tmem_ld_wait();
          if (whole) {
            if (dst && !dead)
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t x[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  x[k] = l == 0.0f ? 0u
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
            kp_tiles(p.part)[cta] = KpTile{own.y - own.x + 1, sg.t, sg.g, sg.s.off, sg.s.n, {0, 0, 0}};
        }
        ++seg;
      }
      if (tid == 0) s_n[seg & 1] = 0;      // no more segments
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
        if (w > w_beg && w < w_end) kv8_next<KP_U, KP_COST>(sg, p, prefix, w, w_end);
        const bool more = w < w_end;
        const int end = kv8_seg_end(sg, p.tq_shift);
        const int* table = p.b.page_table + static_cast<size_t>(sg.b) * p.b.max_pages;
        int u = more ? sg.u0 : 0;
        const int u1 = more ? sg.u1 : 1;               // at the end one more plan: no more tiles
        int pid = -1;
        const auto look = [&] {
          const int pos = u * KP_U + lb * KV8_BLOCK;
          pid = more && u < u1 && pos < end ? __ldg(table + (pos >> p.c.page_shift)) : -1;
        };
        look();
#pragma unroll 1
        while (u < u1) {
          const int pos = u * KP_U + lb * KV8_BLOCK;
          const bool exists = more && pos < end, bad = exists && (pid < 0 || pid >= p.c.n_pages);
          int row = -1;
          float scale = 0.0f;
          if (exists && !bad) {
            row = ((pid * p.c.hkv + sg.g) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1));   // below 2^31
            scale = __ldg(p.c.scales[(lane >> 3) & 1] + row / KV8_BLOCK);
          }
          // A sequence with fewer positions than new tokens has units past its end: nothing valid
          // in them, which is not the mark of the end.
          const int valid = more ? max(end - u * KP_U, 0) : -1;
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

// ---------------------------------------------------------------- host side
size_t kv8_prompt_ws_bytes(int D) {
  return KV8_TICKET_BYTES + KP_TILES_BYTES +
         static_cast<size_t>(KV8_MAX_CTAS) * 2 * (2 * KP_ROWS) * kp_ps(D) * sizeof(float);
}

namespace {
template <int D, int FMT>
cudaError_t launch_prompt(const Kv8AttnParams& p, int nblk, int grid, int dev, cudaStream_t s) {
  static bool set[KV8_MAX_DEVICES] = {};
  auto* k = kv8_prompt_kernel<D, FMT>;
  if (!set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kp_smem(D, KV8_MAX_SEQS));
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  const cudaError_t e = launch_pdl(k, dim3(grid), dim3(KP_THREADS), kp_smem(D, p.b.n_seqs), s, p, nblk);
  if (e != cudaSuccess) return e;
  return launch_pdl(kv8_prompt_join_kernel<D>, dim3(grid, nblk * KP_ROWS / 8), dim3(256), 0, s, p, nblk);
}
}  // namespace

cudaError_t launch_kv8_prompt(Kv8AttnParams p, int D, int format, int grid, int dev, cudaStream_t s) {
  // tokens of a row block: the largest power of two whose rows fit
  int shift = 0;
  while ((2 << shift) * p.G <= KP_ROWS) ++shift;
  const int nblk = p.b.max_new <= (1 << shift) ? 1 : 2;
  p.tq_shift = shift + nblk - 1;
  const bool e4 = format == GQA_KV8_E4M3;
  if (D == 128)
    return e4 ? launch_prompt<128, GQA_KV8_E4M3>(p, nblk, grid, dev, s) : launch_prompt<128, GQA_KV8_INT8>(p, nblk, grid, dev, s);
  return e4 ? launch_prompt<64, GQA_KV8_E4M3>(p, nblk, grid, dev, s) : launch_prompt<64, GQA_KV8_INT8>(p, nblk, grid, dev, s);
}

}  // namespace moe
