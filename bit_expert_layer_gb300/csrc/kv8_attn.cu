// kv8_attn.cu -- attention over the 8-bit key/value cache: the entry points, and the kernel
// for few query rows per key/value head (decode, a few drafted tokens).
//
// Each of a CTA's 8 warps takes a run of the line of its own (pieces of 32 positions) and
// works alone: it streams its pieces (codes of 32 keys and values, TMA boxes with the row's
// swizzle) through a ring of its own, writes out the tiles that lie whole in its run, and
// leaves the two parts at the run's ends in shared memory for the CTA to join at the end, so
// the warps meet once per launch.  (A CTA per tile, joined tile by tile, measured 122 us on
// 64 sequences of 64 to 16384 positions: the short ones cost a barrier round each.)
// Per piece, on mma.sync, R query rows (8 or 16) on the M side:
//   S = Q K^T     fp16 with exact operands: codes are exact in fp16, and a query row is
//                 scaled by a power of two to fit.  The order of the contraction is free, so
//                 a lane takes 32 consecutive dims of a key, one or two 16-byte loads.
//   weights       in base 2, with the value block's scale folded in: w_i = 2^(s_i + e_i - m)
//                 for values of scale 2^e_i, m the running maximum of s_i + e_i.  The value
//                 product takes fp16(w_i) and the bare codes, the normaliser sums
//                 w_i 2^-e_i in fp32; so the scales cost one fused multiply-add per score.
//   O += w V      a lane takes 16 consecutive dims of 4 keys and interleaves their bytes, so
//                 that a pair of codes of one dim becomes an fp16 pair; column n of the
//                 MMA's j-th block is dim 16 n + j.
// Bound: the cache's bytes.  Per 32 positions and SM (8 KB, about 350 cycles at the measured
// copy rate) a warp issues about 350 instructions, spread over 4 schedulers.
#include <cstring>

#include "internal.h"
#include "kv8_host.h"
#include "kv8_sched.cuh"

namespace moe {

namespace {

constexpr int KA_WARPS = 8;
constexpr int KA_THREADS = KA_WARPS * 32;
constexpr int KA_U = 32;                       // positions per piece
constexpr int KA_STAGES = 2;                   // pieces in flight per warp
constexpr int KA_COST = 2;                     // a tile's start, in pieces
__host__ __device__ constexpr int ka_half(int D) { return KA_U * D; }       // bytes of a piece's keys (or values)
__host__ __device__ constexpr int ka_ring(int D) { return KA_WARPS * KA_STAGES * 2 * ka_half(D); }
__host__ __device__ constexpr int ka_ps(int D) { return D + 4; }            // floats of a partial row: O, max, sum
// shared memory: rings (1024-aligned), a part per warp (the tile that began before its run;
// the tile that goes on after it takes the warp's own ring, which is done by then), the line,
// what the parts belong to, barriers and words
__host__ __device__ constexpr int ka_parts(int D, int R) { return KA_WARPS * R * ka_ps(D) * 4; }
__host__ __device__ constexpr int ka_wsum(int R) { return R * KV8_MAX_CTAS * 4; }   // weights of a tile's CTAs
__host__ __device__ constexpr int ka_smem(int D, int R, int B) {
  return 1024 + ka_ring(D) + ka_parts(D, R) + ka_wsum(R) + (B + 2) * 8 + KA_WARPS * (8 + KA_STAGES * 8 + 2 * 32) + 64;
}
static_assert(ka_smem(128, 16, KV8_MAX_SEQS) <= 232448, "shared memory per CTA exceeds 227 KB");
static_assert(16 * ka_ps(128) * 4 <= KA_STAGES * 2 * ka_half(128) && 16 * ka_ps(64) * 4 <= KA_STAGES * 2 * ka_half(64),
              "a warp's part fits its ring");

// What a part belongs to.
struct __align__(16) KaPart {
  int b, g, t;           // sequence, key/value head, tile; b < 0: no part
  int off, n;            // the sequence's first row and new tokens
  int r_first, r_last;   // the runs of the tile's first and last unit
  int pad;
};

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Shared-memory offset of 16-byte chunk c of row r (rows of D bytes, the tensor map's swizzle).
template <int D>
__device__ __forceinline__ uint32_t code_off(int r, int c) {
  if (D == 128) return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// One 16-position block of a piece: bad or past the tile's end when scale < 0.
constexpr float KA_NO_BLOCK = -1.0f;

}  // namespace

// box: rows of the tensor maps' box, 16 (pages of 16 positions) or 32.
template <int D, int R, int FMT>
__global__ void __launch_bounds__(KA_THREADS, 1)
    kv8_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ Kv8AttnParams p, int box) {
  constexpr int NJ = D / 16;          // MMAs of a score block's contraction
  constexpr int ND = D / 8;           // 8-column blocks of O
  constexpr int LD = D / 4;           // dims of a row that a lane's quad member holds
  constexpr int PS = ka_ps(D);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* heads = reinterpret_cast<float*>(smem + ka_ring(D));
  float* wsum = heads + ka_parts(D, R) / 4;
  long long* prefix = reinterpret_cast<long long*>(wsum + ka_wsum(R) / 4);
  long long* s_warp = prefix + p.b.n_seqs + 1 + ((p.b.n_seqs + 1) & 1);      // 16-byte aligned
  KaPart* meta = reinterpret_cast<KaPart*>(s_warp + KA_WARPS);             // [warp][began before, goes on]
  uint64_t* bars = reinterpret_cast<uint64_t*>(meta + 2 * KA_WARPS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + KA_WARPS * KA_STAGES);
  int* s_last = const_cast<int*>(abort_flag) + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g4 = lane >> 2, c4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * KA_STAGES * 2 * ka_half(D);
  const uint32_t bar0 = smem_u32(bars) + warp * KA_STAGES * 8;

  if (tid == 0) {
    for (int i = 0; i < KA_WARPS * KA_STAGES; ++i) mbar_init(smem_u32(bars) + 8 * i, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (tid < 2 * KA_WARPS) meta[tid].b = -1;
  Kv8Runs runs;
  runs.total = kv8_line<KA_U, KA_COST, KA_THREADS>(p, prefix, s_warp);
  runs.n = static_cast<int>(min(runs.total, static_cast<long long>(gridDim.x) * KA_WARPS));
  const int cta = blockIdx.x, run = cta * KA_WARPS + warp;
  if (cta * KA_WARPS >= runs.n) return;
  const long long w_beg = run < runs.n ? kv8_run_begin(runs, run) : 0;
  const long long w_end = run < runs.n ? kv8_run_begin(runs, run + 1) : 0;

  // ---- this warp's load cursor: its next piece, and per lane 0..3 the page of one of the
  // piece's blocks (lane & 1: block, lane >> 1: keys or values)
  long long lw = w_beg;
  Kv8Seg ls = {};
  int lu = 0, l_end = 0, pid = -1;
  bool more = w_beg < w_end;
  if (more) {
    ls = kv8_seg<KA_U, KA_COST>(p, prefix, lw, w_end, runs);
    lu = ls.u0;
    l_end = kv8_seg_end(ls, p.tq_shift);
  }
  const Kv8Seg first_seg = ls;
  auto settle = [&] {                 // the cursor's next piece: its segment and its pages
    if (!more) return;
    while (lu >= ls.u1) {
      lw += ls.len;
      if (lw >= w_end) {
        more = false;
        return;
      }
      kv8_next<KA_U, KA_COST>(ls, p, prefix, lw, w_end, runs);
      lu = ls.u0;
      l_end = kv8_seg_end(ls, p.tq_shift);
    }
    const int pos = lu * KA_U + (lane & 1) * KV8_BLOCK;
    pid = -1;
    if (lane < 4 && pos < l_end)
      pid = __ldg(p.b.page_table + static_cast<size_t>(ls.b) * p.b.max_pages + (pos >> p.c.page_shift));
  };
  const uint64_t pol = l2_policy_evict_first();
  int issued = 0;
  // Issue the cursor's piece into its stage; returns this lane's block scale (lanes 0..3).
  auto issue = [&]() -> float {
    float sc = KA_NO_BLOCK;
    if (!more) return sc;
    const int st = issued % KA_STAGES;
    const int pos = lu * KA_U + (lane & 1) * KV8_BLOCK;
    bool live = lane < 4 && pos < l_end;
    if (live && (pid < 0 || pid >= p.c.n_pages)) {
      atomicOr(p.c.err, ERRBIT_BOUNDS);
      live = false;
    }
    size_t row = 0;
    if (live) {
      row = ((static_cast<size_t>(pid) * p.c.hkv + ls.g) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1));
      sc = fmaxf(__ldg(p.c.scales[lane >> 1] + row / KV8_BLOCK), 0.0f);
    }
    const bool copies = live && (box == KV8_BLOCK || (lane & 1) == 0);   // a box of 32 rows brings both blocks
    const unsigned n = __popc(__ballot_sync(0xffffffffu, copies));
    const uint32_t bar = bar0 + 8 * st;
    if (lane == 0) mbar_arrive_expect_tx(bar, n * box * D);
    __syncwarp();
    if (copies) {
      const uint32_t dst = ring + st * 2 * ka_half(D) + (lane >> 1) * ka_half(D) + (lane & 1) * KV8_BLOCK * D;
      tma_load_2d_hint(dst, lane >> 1 ? &tm_v : &tm_k, bar, 0, static_cast<int>(row), pol);
    }
    ++issued;
    ++lu;
    settle();
    return sc;
  };

  settle();
  float sc_next[KA_STAGES];
#pragma unroll
  for (int i = 0; i < KA_STAGES; ++i) sc_next[i] = issue();

  int taken = 0;
  bool dead = false;      // a wait gave up: nothing more is loaded or computed
  Kv8Seg sg = first_seg;
  for (long long w = w_beg; w < w_end;) {
    if (w > w_beg) kv8_next<KA_U, KA_COST>(sg, p, prefix, w, w_end, runs);
    w += sg.len;
    if (sg.u1 <= sg.u0) continue;     // the run ends before the tile's first piece
    const int end = kv8_seg_end(sg, p.tq_shift);
    const int tok0 = sg.t << p.tq_shift;
    const int ntok = min(1 << p.tq_shift, sg.s.n - tok0);
    const int nrows = ntok * p.G;
    // ---- query fragments: rows g4 and g4 + 8, dims LD c4 ..
    uint32_t qa[2][NJ][2];            // [row half][MMA][register]
    float rs[2];
    int see[2];                       // positions that the row's token sees
#pragma unroll
    for (int h = 0; h < R / 8; ++h) {
      const int r = g4 + 8 * h;
      const int tok = r / p.G, hh = r - tok * p.G;
      uint4 v[LD / 8];
#pragma unroll
      for (int i = 0; i < LD / 8; ++i) v[i] = make_uint4(0, 0, 0, 0);
      see[h] = 0;
      if (r < nrows) {
        const __nv_bfloat16* src =
            p.q + static_cast<size_t>(sg.s.off + tok0 + tok) * p.q_stride + (sg.g * p.G + hh) * D + LD * c4;
#pragma unroll
        for (int i = 0; i < LD / 8; ++i) v[i] = ldg_nc_v4(src + 8 * i);
        see[h] = sg.s.first + tok0 + tok + 1;
      }
      uint32_t big = 0;
#pragma unroll
      for (int i = 0; i < LD / 8; ++i) {
        const uint32_t* x = &v[i].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) big = max(big, max(x[j] & 0x7FFFu, (x[j] >> 16) & 0x7FFFu));
      }
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // the row's largest magnitude lands in [2^13, 2^14): bf16's 8 bits stay exact in fp16
      // down to 2^-28 of it
      const int e = min(max(static_cast<int>(big >> 7) - 127 - 13, -100), 100);
      const float f = pow2i(-e);
      rs[h] = pow2i(e) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint32_t* x = &v[j >> 1].x + (j & 1) * 2;
        qa[h][j][0] = pack2_f16(bf16lo(x[0]) * f, bf16hi(x[0]) * f);
        qa[h][j][1] = pack2_f16(bf16lo(x[1]) * f, bf16hi(x[1]) * f);
      }
    }
    if (R == 8) {
      rs[1] = 0.0f;
      see[1] = 0;
    }
    float m_run[2] = {-INFINITY, -INFINITY}, l_part[2] = {0.0f, 0.0f};
    float o[ND][4];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

    for (int u = sg.u0; u < sg.u1 && !dead; ++u) {
      const int st = taken % KA_STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait(bar0 + 8 * st, (taken / KA_STAGES) & 1, p.c.err, abort_flag, p.wait_ns))) {
        dead = true;
        break;
      }
      ++taken;
      const uint32_t kb = ring + st * 2 * ka_half(D), vb = kb + ka_half(D);
      const float sc = sc_next[0];
      float ksc[2], vsc[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        ksc[i] = __shfl_sync(0xffffffffu, sc, i);
        vsc[i] = __shfl_sync(0xffffffffu, sc, 2 + i);
      }
      // ---- scores of the piece's 4 blocks of 8 keys
      float x[4][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        x[nb][0] = x[nb][1] = x[nb][2] = x[nb][3] = 0.0f;
        if (ksc[nb >> 1] < 0.0f || vsc[nb >> 1] < 0.0f) continue;
        const int r = 8 * nb + g4;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 kv = lds128(kb + code_off<D>(r, (D / 64) * c4 + i));
          const uint32_t* kw = &kv.x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t wd = kv8_flip<FMT>(kw[j]);
            const int jj = 4 * i + j;
            mma_f16_16816(x[nb], qa[0][jj][0], R == 16 ? qa[1][jj][0] : 0u, qa[0][jj][1], R == 16 ? qa[1][jj][1] : 0u,
                          kv8_half2<FMT>(wd, 0), kv8_half2<FMT>(wd, 1));
          }
        }
      }
      // ---- s_i + e_i in base 2, masked; running maximum
      int ve[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) ve[i] = max(scale_exp(vsc[i]), KV8_MIN_EXP);
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        const bool live = !(ksc[nb >> 1] < 0.0f || vsc[nb >> 1] < 0.0f);
        const int pos = u * KA_U + 8 * nb + 2 * c4;
        const float add = static_cast<float>(ve[nb >> 1]);
#pragma unroll
        for (int i = 0; i < (R == 16 ? 4 : 2); ++i) {
          const int h = i >> 1;
          const bool ok = live && pos + (i & 1) < see[h];
          x[nb][i] = ok ? fmaf(x[nb][i] * rs[h], ksc[nb >> 1], add) : -INFINITY;
          mx[h] = fmaxf(mx[h], x[nb][i]);
        }
      }
      uint32_t pa[4][2];              // weights of key pairs: [8-key block][row half]
#pragma unroll
      for (int h = 0; h < R / 8; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        const float m_new = fmaxf(m_run[h], mx[h]);
        const float m_at = m_new == -INFINITY ? 0.0f : m_new;   // no key so far: every weight is 0
        const float corr = exp2f(m_run[h] - m_at);
        m_run[h] = m_new;
        float l = l_part[h] * corr;
#pragma unroll
        for (int nb = 0; nb < 4; ++nb) {
          const float w0 = exp2f(x[nb][2 * h] - m_at), w1 = exp2f(x[nb][2 * h + 1] - m_at);
          l = fmaf(w0 + w1, pow2i(-ve[nb >> 1]), l);
          pa[nb][h] = pack2_f16(w0, w1);
        }
        l_part[h] = l;
#pragma unroll
        for (int i = 0; i < ND; ++i) {
          o[i][2 * h] *= corr;
          o[i][2 * h + 1] *= corr;
        }
      }
      // ---- O += w V, 16 keys a step; rows past the tile's end are not looked at
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        if (ksc[ks] < 0.0f || vsc[ks] < 0.0f) continue;
        const int r = 16 * ks + 2 * c4;
        constexpr int W = D / 32;     // words of a row per lane
        uint32_t rw[4][W];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = r + (i & 1) + (i >> 1) * 8;
          if (D == 128) {
            const uint4 v = lds128(vb + code_off<D>(rr, g4));
            rw[i][0] = v.x, rw[i][1] = v.y, rw[i][W - 2] = v.z, rw[i][W - 1] = v.w;
          } else {
            const uint2 v = lds64(vb + code_off<D>(rr, g4 >> 1) + (g4 & 1) * 8);
            rw[i][0] = v.x, rw[i][1] = v.y;
          }
        }
        const int base = u * KA_U + 16 * ks;
        if (base + 16 > end) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + 2 * c4 + (i & 1) + (i >> 1) * 8 >= end)
#pragma unroll
              for (int j = 0; j < W; ++j) rw[i][j] = 0;
        }
        const uint32_t a0 = pa[2 * ks][0], a2 = pa[2 * ks + 1][0];
        const uint32_t a1 = R == 16 ? pa[2 * ks][1] : 0u, a3 = R == 16 ? pa[2 * ks + 1][1] : 0u;
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t lo01 = kv8_flip<FMT>(__byte_perm(rw[0][j], rw[1][j], 0x5140));
          const uint32_t hi01 = kv8_flip<FMT>(__byte_perm(rw[0][j], rw[1][j], 0x7362));
          const uint32_t lo23 = kv8_flip<FMT>(__byte_perm(rw[2][j], rw[3][j], 0x5140));
          const uint32_t hi23 = kv8_flip<FMT>(__byte_perm(rw[2][j], rw[3][j], 0x7362));
          mma_f16_16816(o[4 * j + 0], a0, a1, a2, a3, kv8_half2<FMT>(lo01, 0), kv8_half2<FMT>(lo23, 0));
          mma_f16_16816(o[4 * j + 1], a0, a1, a2, a3, kv8_half2<FMT>(lo01, 1), kv8_half2<FMT>(lo23, 1));
          mma_f16_16816(o[4 * j + 2], a0, a1, a2, a3, kv8_half2<FMT>(hi01, 0), kv8_half2<FMT>(hi23, 0));
          mma_f16_16816(o[4 * j + 3], a0, a1, a2, a3, kv8_half2<FMT>(hi01, 1), kv8_half2<FMT>(hi23, 1));
        }
      }
      // the stage is free once every lane has read it
      __syncwarp();
#pragma unroll
      for (int i = 0; i + 1 < KA_STAGES; ++i) sc_next[i] = sc_next[i + 1];
      sc_next[KA_STAGES - 1] = issue();
    }

    // ---- the tile's rows: out if the whole tile lies in this run, else a part for the CTA
    const bool whole = sg.u0 == 0 && sg.u1 == sg.units;
#pragma unroll
    for (int h = 0; h < R / 8; ++h) {
      float l = l_part[h];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int r = g4 + 8 * h;
      // block j holds dim (D / 8) n + j of columns n = 2 c4, 2 c4 + 1: this lane's LD dims
      if (whole) {
        if (r < nrows) {
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;   // a row that saw no key: zeros
          const int tok = r / p.G, hh = r - tok * p.G;
          __nv_bfloat16* dst =
              p.out + (static_cast<size_t>(sg.s.off + tok0 + tok) * p.hq + sg.g * p.G + hh) * D + LD * c4;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < ND; j += 8) {
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                x[k] = pack_bf16x2(__float_as_uint(o[j + 2 * k][2 * h + i] * inv),
                                   __float_as_uint(o[j + 2 * k + 1][2 * h + i] * inv));
              *reinterpret_cast<uint4*>(dst + ND * i + j) = make_uint4(x[0], x[1], x[2], x[3]);
            }
        }
      } else {
        if (sg.u0 == 0) __syncwarp();   // the ring: every lane has read its last piece
        float* row = (sg.u0 ? heads + warp * R * PS
                            : reinterpret_cast<float*>(smem + warp * KA_STAGES * 2 * ka_half(D))) + r * PS;
        if (c4 == 0) {
          row[D] = m_run[h];
          row[D + 1] = l;
        }
        float* dst = row + LD * c4;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < ND; j += 4)
            *reinterpret_cast<float4*>(dst + ND * i + j) =
                make_float4(o[j][2 * h + i], o[j + 1][2 * h + i], o[j + 2][2 * h + i], o[j + 3][2 * h + i]);
      }
    }
    if (!whole && lane == 0)
      meta[2 * warp + (sg.u0 == 0)] = KaPart{sg.b, sg.g, sg.t, sg.s.off, sg.s.n, sg.w_first, sg.w_last, 0};
  }
  // a warp that gave up: copies still in flight land before the shared memory goes away
  for (; taken < issued; ++taken) {
    const unsigned long long t0 = globaltimer_ns();
    while (!mbar_try_wait(bar0 + 8 * (taken % KA_STAGES), (taken / KA_STAGES) & 1) &&
           globaltimer_ns() - t0 < WAIT_LIMIT_NS) {
    }
  }
  __syncthreads();

  // ---- the parts meet.  A tile's parts in this CTA are the tail of one warp and the heads
  // of the warps after it (or heads from warp 0 on, if it began in an earlier CTA).
  constexpr int TPR = D / 8;                 // threads per row, 8 dims each
  constexpr int ACT = R * TPR;               // 64 .. 256 threads
  const int row = tid / TPR, d0 = (tid % TPR) * 8;
  for (int i0 = -1; i0 < KA_WARPS; ++i0) {
    const KaPart pt = i0 < 0 ? meta[0] : meta[2 * i0 + 1];
    if (pt.b < 0) continue;
    const int last = min(pt.r_last - cta * KA_WARPS, KA_WARPS - 1);   // the tile's last warp here
    const int c_first = pt.r_first / KA_WARPS, c_last = pt.r_last / KA_WARPS;
    const auto part = [&](int i) {           // i0: the tail (or nothing, for -1), above: heads
      return (i == i0 ? reinterpret_cast<const float*>(smem + i * KA_STAGES * 2 * ka_half(D)) : heads + i * R * PS) + row * PS;
    };
    const int i1 = max(i0, 0);
    float M = -INFINITY, L = 0.0f, O[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (tid < ACT) {
      for (int i = i1; i <= last; ++i) M = fmaxf(M, part(i)[D]);
      const float at = M == -INFINITY ? 0.0f : M;
      for (int i = i1; i <= last; ++i) {
        const float* src = part(i);
        const float f = exp2f(src[D] - at);
        L = fmaf(f, src[D + 1], L);
#pragma unroll
        for (int k = 0; k < 8; ++k) O[k] = fmaf(f, src[d0 + k], O[k]);
      }
    }
    bool write = c_first == c_last;
    if (!write) {
      const auto slot = [&](int c) { return p.part + ((static_cast<size_t>(c) * 2 + (c == c_first)) * R + row) * PS; };
      if (tid < ACT) {
        float* dst = slot(cta);
        *reinterpret_cast<float4*>(dst + d0) = make_float4(O[0], O[1], O[2], O[3]);
        *reinterpret_cast<float4*>(dst + d0 + 4) = make_float4(O[4], O[5], O[6], O[7]);
        if (d0 == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(M, L);
      }
      __threadfence();
      __syncthreads();
      const int ns = c_last - c_first + 1;
      if (tid == 0) {
        const bool all = atomicAdd(p.tickets + c_first, 1u) == static_cast<unsigned>(ns) - 1u;
        if (all) p.tickets[c_first] = 0u;    // every part has arrived: ready for the next call
        *s_last = all;
      }
      __syncthreads();
      write = *s_last != 0;
      if (write) {
        __threadfence();
        float* fs = wsum;                    // [R][ns] weights of the CTAs' sums, in the order of the line
        L = 0.0f;
        if (tid < ACT) {
          const int j0 = tid % TPR;
          M = -INFINITY;
          for (int i = j0; i < ns; i += TPR) M = fmaxf(M, __ldcg(slot(c_first + i) + D));
#pragma unroll
          for (int s = TPR / 2; s >= 1; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
          const float at = M == -INFINITY ? 0.0f : M;
          for (int i = j0; i < ns; i += TPR) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(slot(c_first + i) + D));
            const float f = exp2f(ml.x - at);
            L = fmaf(f, ml.y, L);
            fs[row * ns + i] = f;
          }
#pragma unroll
          for (int s = TPR / 2; s >= 1; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
        }
        __syncthreads();
        if (tid < ACT) {
#pragma unroll
          for (int k = 0; k < 8; ++k) O[k] = 0.0f;
#pragma unroll 4
          for (int i = 0; i < ns; ++i) {
            const float f = fs[row * ns + i];
            const float4 a = __ldcg(reinterpret_cast<const float4*>(slot(c_first + i) + d0));
            const float4 b = __ldcg(reinterpret_cast<const float4*>(slot(c_first + i) + d0 + 4));
            O[0] = fmaf(f, a.x, O[0]), O[1] = fmaf(f, a.y, O[1]), O[2] = fmaf(f, a.z, O[2]), O[3] = fmaf(f, a.w, O[3]);
            O[4] = fmaf(f, b.x, O[4]), O[5] = fmaf(f, b.y, O[5]), O[6] = fmaf(f, b.z, O[6]), O[7] = fmaf(f, b.w, O[7]);
          }
        }
      }
    }
    const int tok0 = pt.t << p.tq_shift;
    if (write && tid < ACT && row < min(1 << p.tq_shift, pt.n - tok0) * p.G) {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;   // a row that saw no key: zeros
      const int tok = row / p.G, hh = row - tok * p.G;
      uint4 r;
      r.x = pack_bf16x2(__float_as_uint(O[0] * inv), __float_as_uint(O[1] * inv));
      r.y = pack_bf16x2(__float_as_uint(O[2] * inv), __float_as_uint(O[3] * inv));
      r.z = pack_bf16x2(__float_as_uint(O[4] * inv), __float_as_uint(O[5] * inv));
      r.w = pack_bf16x2(__float_as_uint(O[6] * inv), __float_as_uint(O[7] * inv));
      *reinterpret_cast<uint4*>(p.out + (static_cast<size_t>(pt.off + tok0 + tok) * p.hq + pt.g * p.G + hh) * D + d0) = r;
    }
  }
}

// ============================================================================ C ABI
namespace {

// Largest power of two that is at most n (n >= 1), as a shift.
int floor_log2(int n) {
  int s = 0;
  while ((2 << s) <= n) ++s;
  return s;
}

// Query rows of a tile: 8 or 16 when the group's rows of all new tokens fit, else 0 (the
// prompt kernel).
int ka_rows(int G, int max_new) {
  const long long n = static_cast<long long>(G) * max_new;
  return n <= 8 ? 8 : n <= 16 ? 16 : 0;
}

size_t kv8_ws_bytes(int D, int rows) {
  if (!rows) return kv8_prompt_ws_bytes(D);
  return KV8_TICKET_BYTES + static_cast<size_t>(KV8_MAX_CTAS) * 2 * rows * ka_ps(D) * sizeof(float);
}

template <int D, int R, int FMT>
cudaError_t launch_decode(const CUtensorMap& tk, const CUtensorMap& tv, const Kv8AttnParams& p, int box, int grid, int dev,
                          cudaStream_t s) {
  static bool set[KV8_MAX_DEVICES] = {};
  auto* k = kv8_decode_kernel<D, R, FMT>;
  if (!set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ka_smem(D, R, KV8_MAX_SEQS));
    if (e != cudaSuccess) return e;
    set[dev] = true;
  }
  k<<<grid, KA_THREADS, ka_smem(D, R, p.b.n_seqs), s>>>(tk, tv, p, box);
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" size_t gqa_kv8_workspace_bytes(const gqa_kv8_cache_t* cache, int n_q_heads, int max_new) {
  if (!cache || (cache->head_size != 64 && cache->head_size != 128) || cache->n_kv_heads < 1 || max_new < 1 ||
      max_new > (1 << 20) || n_q_heads < 1 || n_q_heads % cache->n_kv_heads || n_q_heads / cache->n_kv_heads > 16)
    return 0;
  return kv8_ws_bytes(cache->head_size, ka_rows(n_q_heads / cache->n_kv_heads, max_new));
}

extern "C" moe_status_t gqa_kv8_attention(const gqa_kv8_cache_t* cache, const gqa_kv8_batch_t* batch, const void* q,
                                          long long q_stride, int n_q_heads, float scale, void* out, void* workspace,
                                          size_t workspace_bytes, moe_stream_t stream) {
  moe_status_t st;
  if (!kv8_cache_ok(cache, &st) || !kv8_batch_ok(cache, batch, &st)) return st;
  if (n_q_heads < 1 || !workspace || !(scale >= 0.0f && scale <= 1e30f)) return MOE_ERR_INVALID_ARG;
  if (n_q_heads % cache->n_kv_heads || n_q_heads / cache->n_kv_heads > 16) return MOE_ERR_UNSUPPORTED;
  const int D = cache->head_size;
  const long long width = static_cast<long long>(n_q_heads) * D;
  if (batch->n_tokens == 0) return MOE_OK;
  if (!kv8_rows_ok(q, q_stride, width, &st) || !kv8_rows_ok(out, width, width, &st)) return st;
  if (reinterpret_cast<uintptr_t>(workspace) & 255u) return MOE_ERR_ALIGNMENT;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  const uintptr_t qn = 2 * (static_cast<uintptr_t>(batch->n_tokens - 1) * q_stride + width);
  if (q0 < o0 + 2 * static_cast<uintptr_t>(batch->n_tokens) * width && o0 < q0 + qn) return MOE_ERR_INVALID_ARG;
  const int G = n_q_heads / cache->n_kv_heads, R = ka_rows(G, batch->max_new);
  if (workspace_bytes < kv8_ws_bytes(D, R)) return MOE_ERR_WORKSPACE;

  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && (dev < 0 || dev >= KV8_MAX_DEVICES)) e = cudaErrorInvalidDevice;
  static int sm_count[KV8_MAX_DEVICES] = {};
  if (e == cudaSuccess && !sm_count[dev]) {
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) sm_count[dev] = sms;
  }
  if (e != cudaSuccess) {
    set_error_detail("gqa_kv8_attention: device", e);
    return MOE_ERR_CUDA;
  }
  const int grid = sm_count[dev] < KV8_MAX_CTAS ? sm_count[dev] : KV8_MAX_CTAS;

  Kv8AttnParams p;
  std::memset(&p, 0, sizeof p);
  p.c = kv8_cache(cache);
  p.b = kv8_batch(batch);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.out_wide = (o0 & 31u) == 0;
  p.hq = n_q_heads;
  p.G = G;
  p.tq_shift = R ? floor_log2(R / G) : 0;
  p.scale_log2 = (scale > 0.0f ? scale : 1.0f / sqrtf(static_cast<float>(D))) * 1.4426950408889634f;
  p.tickets = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + KV8_TICKET_BYTES);
  p.wait_ns = wait_limit_ns();

  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (!R) {
    e = launch_kv8_prompt(p, D, cache->format, grid, dev, s);
    if (e != cudaSuccess) {
      set_error_detail("gqa_kv8_attention: launch", e);
      return MOE_ERR_CUDA;
    }
    return MOE_OK;
  }
  CUtensorMap tk, tv;
  const uint64_t rows = static_cast<uint64_t>(cache->n_pages) * cache->n_kv_heads * cache->page_size;
  const int box = cache->page_size >= KA_U ? KA_U : KV8_BLOCK;
  if (!encode_u8_rows(&tk, cache->k_codes, D, rows, box) || !encode_u8_rows(&tv, cache->v_codes, D, rows, box))
    return MOE_ERR_CUDA;
  const bool e4 = cache->format == GQA_KV8_E4M3;
  if (D == 128 && R == 8)
    e = e4 ? launch_decode<128, 8, GQA_KV8_E4M3>(tk, tv, p, box, grid, dev, s)
           : launch_decode<128, 8, GQA_KV8_INT8>(tk, tv, p, box, grid, dev, s);
  else if (D == 128)
    e = e4 ? launch_decode<128, 16, GQA_KV8_E4M3>(tk, tv, p, box, grid, dev, s)
           : launch_decode<128, 16, GQA_KV8_INT8>(tk, tv, p, box, grid, dev, s);
  else if (R == 8)
    e = e4 ? launch_decode<64, 8, GQA_KV8_E4M3>(tk, tv, p, box, grid, dev, s)
           : launch_decode<64, 8, GQA_KV8_INT8>(tk, tv, p, box, grid, dev, s);
  else
    e = e4 ? launch_decode<64, 16, GQA_KV8_E4M3>(tk, tv, p, box, grid, dev, s)
           : launch_decode<64, 16, GQA_KV8_INT8>(tk, tv, p, box, grid, dev, s);
  if (e != cudaSuccess) {
    set_error_detail("gqa_kv8_attention: launch", e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
