// kv8_prompt.cu -- attention over the 8-bit key/value cache for many query rows per
// key/value head (prompts, pieces of one, more drafted tokens than the decode kernel's 16
// rows hold), on tcgen05.
//
// A CTA works on one or two blocks of 128 query rows (TQ tokens x G heads each) that share
// their keys, in tiles of 128 positions; its 16 warps have roles:
//   warps 0-7    softmax, one query row per thread, four warps per row block
//   warps 8-11   dequantise: codes from global memory into fp16 tiles in shared memory,
//                128-byte rows with the 128-byte swizzle, two buffers each for K and V
//   warp 12      issues the MMAs
// Per tile and row block, TMEM lane = query row:
//   S = Q K^T    both operands in shared memory.  fp16 holds every code exactly, and a query
//                row is scaled by a power of two to fit, so the products are exact.
//   softmax      in base 2 with the value block's scale folded in, as in the decode kernel:
//                w_i = 2^(s_i + e_i - m), normaliser sum w_i 2^-e_i in fp32.  The reference m
//                moves only when the maximum has grown by more than 2^8: until then weights
//                up to 2^8 fit fp16 as exactly as smaller ones, and O in TMEM needs no
//                rescaling.  fp16(w) goes back to TMEM over S.
//   O += w V     w from TMEM, V from shared memory, its rows as they are (N-major operand)
// The two row blocks alternate: while one is in its softmax the tensor cores work for the
// other (order of issue: PV of block 0, next QK of block 0, PV of block 1, next QK of block 1).
// Bound: per tile and two row blocks 16.8 MFLOP of MMA (2048 cycles at the nominal rate), and
// 32768 exponentials.
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "kv8_host.h"
#include "kv8_sched.cuh"

namespace moe {

namespace {

constexpr int KP_THREADS = 512;
constexpr int KP_U = 128;                         // positions per tile
constexpr int KP_ROWS = 128;                      // query rows per block
constexpr int KP_NB = KP_U / KV8_BLOCK;           // scales per tile
constexpr int KP_SLOTS = 4;                       // tiles whose scales are kept
constexpr float KP_GROW = 8.0f;                   // the maximum may outgrow the reference by 2^8
__host__ __device__ constexpr int kp_tile(int D) { return KP_U * D * 2; }     // fp16 K or V tile (or 128 query rows)
__host__ __device__ constexpr int kp_smem(int D, int B) {
  // alignment, Q of two blocks, two K and two V tiles, scales, line, scan words, barriers and words
  return 1024 + 6 * kp_tile(D) + KP_SLOTS * 3 * KP_NB * 4 + (B + 2) * 8 + KP_THREADS / 32 * 8 + 16 * 8 + 64;
}
static_assert(kp_smem(128, KV8_MAX_SEQS) <= 232448, "shared memory per CTA exceeds 227 KB");

enum { BAR_KF = 0, BAR_KE = 2, BAR_VF = 4, BAR_VE = 6, BAR_Q = 8, BAR_S = 9, BAR_P = 11, BAR_PV = 13, BAR_END = 15, BAR_N = 16 };

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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t pack2h(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
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
// A tile whose parts lie in several CTAs, left by its first CTA for the kernel that joins them.
struct __align__(16) KpTile {
  int ns;                // CTAs (0: no such tile)
  int t, g, off, n;      // tile, key/value head, the sequence's first row and new tokens
  int pad[3];
};

// Workspace of a part: floats of a row (O, reference, normaliser), the rows of CTA c's part of
// a tile that began in CTA c_first, and the tiles to join, one entry per CTA.
__host__ __device__ constexpr int kp_ps(int D) { return D + 4; }
constexpr size_t KP_TILES_BYTES = KV8_MAX_CTAS * sizeof(KpTile);
__device__ __forceinline__ KpTile* kp_tiles(float* part) { return reinterpret_cast<KpTile*>(part); }
template <int D>
__device__ __forceinline__ float* kp_slot(float* part, int c, int c_first, int row) {
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
  // [slot][8] each: K scale, exponent e of the V scale (-inf: no such block), 2^-e
  float* s_ks = reinterpret_cast<float*>(smem + 6 * TILE);
  float* s_ve = s_ks + KP_SLOTS * KP_NB;
  float* s_vi = s_ve + KP_SLOTS * KP_NB;
  long long* prefix = reinterpret_cast<long long*>(s_vi + KP_SLOTS * KP_NB);
  long long* s_warp = prefix + p.b.n_seqs + 1;
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_warp + KP_THREADS / 32);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + BAR_N);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(const_cast<int*>(abort_flag) + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * i; };

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BAR_KF + i), 4);
      mbar_init(bar(BAR_KE + i), 1);
      mbar_init(bar(BAR_VF + i), 4);
      mbar_init(bar(BAR_VE + i), 1);
      mbar_init(bar(BAR_S + i), 1);
      mbar_init(bar(BAR_P + i), 4);
      mbar_init(bar(BAR_PV + i), 1);
    }
    mbar_init(bar(BAR_Q), 4 * nblk);
    mbar_init(bar(BAR_END), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  Kv8Runs runs;
  runs.total = kv8_line<KP_U, KP_THREADS>(p, prefix, s_warp);
  runs.n = static_cast<int>(min(runs.total, static_cast<long long>(gridDim.x)));
  const int cta = blockIdx.x;
  if (cta >= runs.n) {                          // the whole CTA, before any TMEM is held
    if (tid == 0) kp_tiles(p.part)[cta].ns = 0;
    return;
  }
  const long long w_beg = kv8_run_begin(runs, cta), w_end = kv8_run_begin(runs, cta + 1);
  if (warp == 12) {
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
      int it = 0;
      KpTile tile = {0, 0, 0, 0, 0, {0, 0, 0}};
      Kv8Seg sg = kv8_seg<KP_U>(p, prefix, w_beg, w_end, runs);
      for (long long w = w_beg; w < w_end;) {
        if (w > w_beg) kv8_next<KP_U>(sg, p, prefix, w, w_end, runs);
        const int tok = (sg.t << p.tq_shift) + blk * blk_tokens + r / p.G, hh = r % p.G;
        const bool live = r / p.G < blk_tokens && tok < sg.s.n;
        // positions that the row sees; a row without a token (zeros) needs no mask
        const int see = live ? sg.s.first + tok + 1 : 1 << 30;
        // ---- the query row, scaled into fp16, into the swizzled tile
        float rs;
        {
          const __nv_bfloat16* src = p.q + static_cast<size_t>(sg.s.off + tok) * p.q_stride + (sg.g * p.G + hh) * D;
          uint32_t big = 0;
          if (live)
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = ldg_nc_v4(src + 8 * c);
              const uint32_t* x = &v.x;
#pragma unroll
              for (int j = 0; j < 4; ++j) big = max(big, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
            }
          const int e = min(max(static_cast<int>(big >> 7) - 127 - 13, -100), 100);
          const float f = pow2i(-e);
          rs = pow2i(e) * p.scale_log2;
          uint8_t* dst = s_q + blk * TILE + r * 128;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (live) v = ldg_nc_v4(src + 8 * c);
            uint4 o;
            o.x = pack2h(bf16lo(v.x) * f, bf16hi(v.x) * f);
            o.y = pack2h(bf16lo(v.y) * f, bf16hi(v.y) * f);
            o.z = pack2h(bf16lo(v.z) * f, bf16hi(v.z) * f);
            o.w = pack2h(bf16lo(v.w) * f, bf16hi(v.w) * f);
            *reinterpret_cast<uint4*>(dst + (c >> 3) * BOX + (((c & 7) ^ (r & 7)) << 4)) = o;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(BAR_Q));

        float m_ref = -INFINITY, l = 0.0f;
        for (int u = sg.u0; u < sg.u1; ++u, ++it) {
          wait(BAR_S + blk, it);
          if (dead) continue;
          tc_fence_after();
          const float* ks = s_ks + (it & (KP_SLOTS - 1)) * KP_NB;
          const float* ve = s_ve + (it & (KP_SLOTS - 1)) * KP_NB;
          const float* vi = s_vi + (it & (KP_SLOTS - 1)) * KP_NB;
          const int left = see - u * KP_U;                       // positions of the tile that the row sees
          const bool edge = __any_sync(0xffffffffu, left < KP_U);
          // A tile at the causal edge takes a path of its own (EDGE), so that the others carry
          // no mask: 2 of 5 instructions per score, measured.  The scores are read twice, 32
          // columns at a time, the next ones while these are worked on: 128 of them in
          // registers do not fit beside the rest.
          uint32_t sc[2][32];
          // ---- pass 1: the maximum of s_i + e_i
          float mx = -INFINITY;
          const auto largest = [&](auto edge_c) {
            constexpr bool EDGE = decltype(edge_c)::value;
            tmem_ld32(t_s, sc[0]);
#pragma unroll 1
            for (int c2 = 0; c2 < KP_U / 64; ++c2)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int c = 2 * c2 + k;
                tmem_ld_wait();
                tmem_ld32(t_s + 32 * ((c + 1) & (KP_U / 32 - 1)), sc[k ^ 1]);   // last: pass 2's first
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t* x = sc[k] + 16 * h;
                  const float f = fminf(rs * ks[2 * c + h], 1e37f), e = ve[2 * c + h];
                  if (EDGE) {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                      if (32 * c + 16 * h + j < left) mx = fmaxf(mx, fmaf(__uint_as_float(x[j]), f, e));
                  } else {
                    float m[5];
#pragma unroll
                    for (int j = 0; j < 5; ++j)
                      m[j] = max3(__uint_as_float(x[3 * j]), __uint_as_float(x[3 * j + 1]), __uint_as_float(x[3 * j + 2]));
                    m[0] = max3(m[0], m[1], __uint_as_float(x[15]));
                    m[2] = max3(m[2], m[3], m[4]);
                    mx = fmaxf(mx, fmaf(fmaxf(m[0], m[2]), f, e));
                  }
                }
              }
          };
          if (edge) largest(std::true_type{}); else largest(std::false_type{});
          // ---- the reference moves: O and the normaliser follow
          const bool grow = mx > m_ref + KP_GROW;                // also the first finite maximum
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? mx : m_ref;
            const float corr = grow ? ex2(m_ref - m_new) : 1.0f;   // -inf - finite: 0
            m_ref = m_new;
            l *= corr;
            if (u > sg.u0) {
              wait(BAR_PV + blk, it - 1);
              if (dead) continue;
              tc_fence_after();
#pragma unroll
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
          const float m_at = m_ref == -INFINITY ? 0.0f : m_ref;
          // ---- pass 2: weights, over the scores that were read
          const auto weights = [&](auto edge_c) {
            constexpr bool EDGE = decltype(edge_c)::value;
#pragma unroll 1
            for (int c2 = 0; c2 < KP_U / 64; ++c2)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int c = 2 * c2 + k;
                tmem_ld_wait();
                tmem_ld32(t_s + 32 * ((c + 1) & (KP_U / 32 - 1)), sc[k ^ 1]);   // last: not used
                uint32_t w16[16];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t* x = sc[k] + 16 * h;
                  const float f = fminf(rs * ks[2 * c + h], 1e37f), add = ve[2 * c + h] - m_at;
                  const uint64_t f2 = f32x2(f, f), a2 = f32x2(add, add);
                  uint64_t sum[2] = {0, 0};
#pragma unroll
                  for (int j = 0; j < 8; ++j) {
                    const float2 y = f32x2_get(fma2(f32x2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), f2, a2));
                    float w0 = ex2(y.x), w1 = ex2(y.y);
                    if (EDGE) {
                      if (32 * c + 16 * h + 2 * j >= left) w0 = 0.0f;
                      if (32 * c + 16 * h + 2 * j + 1 >= left) w1 = 0.0f;
                    }
                    sum[j & 1] = add2(sum[j & 1], f32x2(w0, w1));
                    w16[8 * h + j] = pack2h(w0, w1);
                  }
                  const float2 t = f32x2_get(add2(sum[0], sum[1]));
                  l = fmaf(t.x + t.y, vi[2 * c + h], l);
                }
                tmem_st16(t_s + 16 * c, w16);
              }
            tmem_ld_wait();
          };
          if (edge) weights(std::true_type{}); else weights(std::false_type{});
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
        __nv_bfloat16* dst =
            live ? p.out + (static_cast<size_t>(sg.s.off + tok) * p.hq + sg.g * p.G + hh) * D : nullptr;
        float* part = kp_slot<D>(p.part, cta, sg.w_first, blk * KP_ROWS + r);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_o + 32 * c, o);
          tmem_ld_wait();
          if (whole) {
            if (dst && !dead)
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                uint32_t x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  x[k] = l == 0.0f ? 0u
                                   : pack_bf16x2(__float_as_uint(__uint_as_float(o[j + 2 * k]) * inv),
                                                 __float_as_uint(__uint_as_float(o[j + 2 * k + 1]) * inv));
                *reinterpret_cast<uint4*>(dst + 32 * c + j) = make_uint4(x[0], x[1], x[2], x[3]);
              }
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<uint4*>(part + 32 * c + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
        }
        tc_fence_before();
        if (!whole) {
          *reinterpret_cast<float2*>(part + D) = make_float2(m_ref, l);
          if (tid == 0 && sg.w_first == cta) tile = KpTile{sg.w_last - sg.w_first + 1, sg.t, sg.g, sg.s.off, sg.s.n, {0, 0, 0}};
        }
        w += sg.u1 - sg.u0;
      }
      if (tid == 0) kp_tiles(p.part)[cta] = tile;
    }
  } else if (warp < 12) {
    // ================================================ dequantise
    constexpr int CPR = D / 16;                 // 16-byte chunks of codes per row
    constexpr int RPI = 128 / CPR;              // rows per step of the 128 threads
    constexpr int NI = KP_U / RPI;              // steps per tile
    const int dt = tid - 256, cc = dt % CPR, r0 = dt / CPR;
    long long w = w_beg;
    Kv8Seg sg = kv8_seg<KP_U>(p, prefix, w, w_end, runs);
    int u = sg.u0, end = kv8_seg_end(sg, p.tq_shift);
    bool more = true;
    // lane b < 8 of every warp: the page of the cursor's tile's block b, then its code row
    int pid = -1;
    auto look = [&] {
      const int pos = u * KP_U + (lane & 7) * KV8_BLOCK;
      pid = -1;
      if (more && pos < end) {
        pid = __ldg(p.b.page_table + static_cast<size_t>(sg.b) * p.b.max_pages + (pos >> p.c.page_shift));
      }
    };
    auto step = [&] {                           // the cursor's next tile
      if (++u >= sg.u1) {
        w += sg.u1 - sg.u0;
        more = w < w_end;
        if (more) {
          kv8_next<KP_U>(sg, p, prefix, w, w_end, runs);
          u = sg.u0;
          end = kv8_seg_end(sg, p.tq_shift);
        }
      }
      look();
    };
    uint4 kreg[NI], vreg[NI];
    int rows = -1;                              // lane b: first code row of block b (negative: none)
    int valid = 0;                              // positions of the tile before the sequence's end
    float ksc = 0.0f, vex = -INFINITY;
    auto resolve = [&] {                        // the looked-up tile's rows and scales
      const int pos = u * KP_U + (lane & 7) * KV8_BLOCK;
      rows = -1;
      valid = end - u * KP_U;
      ksc = 0.0f;
      vex = -INFINITY;
      if (more && pos < end) {
        if (pid < 0 || pid >= p.c.n_pages) {
          if (lane < 8) atomicOr(p.c.err, ERRBIT_BOUNDS);
        } else {
          rows = ((pid * p.c.hkv + sg.g) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1));   // below 2^31
          ksc = fmaxf(__ldg(p.c.scales[0] + rows / KV8_BLOCK), 0.0f);
          vex = static_cast<float>(max(scale_exp(fmaxf(__ldg(p.c.scales[1] + rows / KV8_BLOCK), 0.0f)), KV8_MIN_EXP));
        }
      }
    };
    auto load = [&](uint4 (&reg)[NI], const uint8_t* codes) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int row = r0 + i * RPI;
        const int at = __shfl_sync(0xffffffffu, rows, row / KV8_BLOCK);
        reg[i] = make_uint4(0, 0, 0, 0);
        if (at >= 0 && row < valid) reg[i] = ldg_nc_v4(codes + static_cast<size_t>(at + row % KV8_BLOCK) * D + 16 * cc);
      }
    };
    auto store = [&](const uint4 (&reg)[NI], uint8_t* tile) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int row = r0 + i * RPI;
        const uint32_t w0 = kv8_flip<FMT>(reg[i].x), w1 = kv8_flip<FMT>(reg[i].y);
        const uint32_t w2 = kv8_flip<FMT>(reg[i].z), w3 = kv8_flip<FMT>(reg[i].w);
        const uint4 a = make_uint4(kv8_half2<FMT>(w0, 0), kv8_half2<FMT>(w0, 1), kv8_half2<FMT>(w1, 0), kv8_half2<FMT>(w1, 1));
        const uint4 b = make_uint4(kv8_half2<FMT>(w2, 0), kv8_half2<FMT>(w2, 1), kv8_half2<FMT>(w3, 0), kv8_half2<FMT>(w3, 1));
        // 8 lanes write one row: the upper box's lanes take their odd chunk first, so that the
        // 8 chunks of a store lie in 8 different bank groups
        uint8_t* dst = tile + (cc >> 2) * BOX + row * 128;
        const int c0 = 2 * (cc & 3), odd = cc >> 2;
        *reinterpret_cast<uint4*>(dst + (((c0 + odd) ^ (row & 7)) << 4)) = odd ? b : a;
        *reinterpret_cast<uint4*>(dst + (((c0 + 1 - odd) ^ (row & 7)) << 4)) = odd ? a : b;
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    look();
    resolve();
    load(kreg, p.c.codes[0]);
    load(vreg, p.c.codes[1]);
    const int tiles = static_cast<int>(w_end - w_beg);
    float ksc_now = ksc, vex_now = vex;
    step();
    for (int it = 0; it < tiles; ++it) {
      const int s = it & 1, ph = (it >> 1) & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(BAR_KE + s), ph ^ 1, p.c.err, abort_flag, p.wait_ns))) break;
      if (warp == 8 && lane < KP_NB) {
        s_ks[(it & (KP_SLOTS - 1)) * KP_NB + lane] = ksc_now;
        s_ve[(it & (KP_SLOTS - 1)) * KP_NB + lane] = vex_now;
        s_vi[(it & (KP_SLOTS - 1)) * KP_NB + lane] = vex_now == -INFINITY ? 0.0f : pow2i(-static_cast<int>(vex_now));
      }
      store(kreg, s_k + s * TILE);
      if (lane == 0) mbar_arrive(bar(BAR_KF + s));
      resolve();
      load(kreg, p.c.codes[0]);
      if (!__all_sync(0xffffffffu, mbar_wait(bar(BAR_VE + s), ph ^ 1, p.c.err, abort_flag, p.wait_ns))) break;
      store(vreg, s_v + s * TILE);
      if (lane == 0) mbar_arrive(bar(BAR_VF + s));
      load(vreg, p.c.codes[1]);
      ksc_now = ksc;
      vex_now = vex;
      step();
    }
  } else if (warp == 12 && lane == 0) {
    // ================================================ MMA issue
    constexpr uint32_t ID_S = idesc_f16(KP_ROWS, KP_U, 0), ID_O = idesc_f16(KP_ROWS, D, 1);
    auto qk = [&](int i, int s) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t a = sdesc_sw128(smem_u32(s_q + i * TILE) + (k >> 2) * BOX) + 2 * (k & 3);
        const uint64_t b = sdesc_sw128(smem_u32(s_k + s * TILE) + (k >> 2) * BOX) + 2 * (k & 3);
        umma_bf16(tmem + 128 * i, a, b, ID_S, k > 0);
      }
      umma_commit(bar(BAR_S + i));
    };
    auto pv = [&](int i, int s, bool acc) {
#pragma unroll
      for (int k = 0; k < KP_U / 16; ++k) {
        const uint64_t b = sdesc_sw128_mn(smem_u32(s_v + s * TILE) + k * 2048, BOX);
        umma_f16_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * k, b, ID_O, acc || k > 0);
      }
      umma_commit(bar(BAR_PV + i));
    };
    auto wait = [&](int b, int phase) {
      const bool ok = mbar_wait(bar(b), phase & 1, p.c.err, abort_flag, p.wait_ns);
      tc_fence_after();
      return ok;
    };
    int it = 0, seg = 0;
    bool ok = true;
    Kv8Seg sg = kv8_seg<KP_U>(p, prefix, w_beg, w_end, runs);
    for (long long w = w_beg; ok && w < w_end; ++seg) {
      if (w > w_beg) kv8_next<KP_U>(sg, p, prefix, w, w_end, runs);
      const int n = sg.u1 - sg.u0;
      ok = wait(BAR_Q, seg) && wait(BAR_KF + (it & 1), it >> 1);
      if (!ok) break;
      for (int i = 0; i < nblk; ++i) qk(i, it & 1);
      umma_commit(bar(BAR_KE + (it & 1)));
      for (int j = 0; ok && j < n; ++j, ++it) {
        const int s = it & 1;
        ok = wait(BAR_VF + s, it >> 1);
        for (int i = 0; ok && i < nblk; ++i) {
          ok = wait(BAR_P + i, it);
          if (!ok) break;
          pv(i, s, j > 0);
          if (i == nblk - 1) umma_commit(bar(BAR_VE + s));
          if (j + 1 < n) {
            if (i == 0) ok = wait(BAR_KF + (s ^ 1), (it + 1) >> 1);
            if (!ok) break;
            qk(i, s ^ 1);
            if (i == nblk - 1) umma_commit(bar(BAR_KE + (s ^ 1)));
          }
        }
      }
      w += n;
    }
    // every MMA issued has to land before the memory goes away
    umma_commit(bar(BAR_END));
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar(BAR_END), 0) && globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
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
  float M = -INFINITY;
  for (int i = lane; i < tl.ns; i += 32) M = fmaxf(M, slot(i)[D]);
#pragma unroll
  for (int s = 16; s >= 1; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  const float at = M == -INFINITY ? 0.0f : M;
  float O[PL], L = 0.0f;
#pragma unroll
  for (int k = 0; k < PL; ++k) O[k] = 0.0f;
#pragma unroll 8
  for (int i = 0; i < tl.ns; ++i) {
    const float* src = slot(i);
    const float2 ml = *reinterpret_cast<const float2*>(src + D);
    const float f = exp2f(ml.x - at);
    L = fmaf(f, ml.y, L);
#pragma unroll
    for (int k = 0; k < PL; k += 2) {
      const float2 v = *reinterpret_cast<const float2*>(src + PL * lane + k);
      O[k] = fmaf(f, v.x, O[k]);
      O[k + 1] = fmaf(f, v.y, O[k + 1]);
    }
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;   // a row that saw no key: zeros
  __nv_bfloat16* dst = p.out + (static_cast<size_t>(tl.off + tok) * p.hq + tl.g * p.G + r - tb * p.G) * D + PL * lane;
#pragma unroll
  for (int k = 0; k < PL; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) = pack_bf16x2(__float_as_uint(O[k] * inv), __float_as_uint(O[k + 1] * inv));
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
  k<<<grid, KP_THREADS, kp_smem(D, p.b.n_seqs), s>>>(p, nblk);
  const cudaError_t e = cudaGetLastError();
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
