// kv8_attn.cu -- attention over the 8-bit key/value cache: the entry points, and the kernel
// for few query rows per key/value head (decode, a few drafted tokens).
//
// Each of a CTA's 8 warps takes a run of the line of its own (pieces of 32 positions) and
// works alone: it streams its pieces (codes of 32 keys and values, TMA boxes with the row's
// swizzle) through a ring of its own, writes out the tiles that lie whole in its run, and
// leaves the two parts at the run's ends in shared memory for the CTA to join at the end, so
// the warps meet once per launch.  (A CTA per tile, joined tile by tile, measured 122 us on
// 64 sequences of 64 to 16384 positions: the short ones cost a barrier round each.)
// Per piece, on mma.sync (m16n8k16, fp16 in, fp32 out), with the R query rows (8 or 16) on the
// N side, so that a full tile of 16 keys or 16 dims meets them:
//   S^T = K Q^T   exact operands: codes are exact in fp16, and a query row is scaled by a power
//                 of two to fit.  The order of the contraction is free, so a lane takes 32
//                 consecutive dims of a key, two 16-byte loads.
//   weights       in base 2, with the value block's scale folded in: w_i = 2^(s_i + e_i - m)
//                 for values of scale 2^e_i, m = ms + d.  The value product takes fp16(w_i) and
//                 the bare codes, the normaliser sums w_i 2^(d - e_i) in fp32; so the scales
//                 cost nothing per score.  The references move only when a row's weights pass
//                 fp16's range at either end, and a piece that does not move them needs little
//                 exchange between lanes.
//   O^T += V^T w  a lane takes 16 consecutive dims of 4 keys and interleaves their bytes, so
//                 that a pair of codes of one dim becomes an fp16 pair; the weights change
//                 from S's layout to B's by a transposing move.
// Bound: the cache's bytes.  8 x 32768 positions of e4m3 (2 heads of 128, 134 MB) take 30 us; a
// plain copy's rate would take 20.  Between its first piece and its last a CTA runs at the
// memory's rate (8 KB per warp and 2400 cycles); 7000 cycles before it (the line, the first
// segment, the first page, the first codes) and 8000 after it (the CTA's join, the ticket, the
// tile's join) are what is left.  With the query rows on the M side (half of each MMA and of O's
// registers empty at 8 rows) a piece took 750 instructions and the same case 36.7 us; 16 warps of
// 16-key pieces took 33.5 us, 12 of three stages 31.8, where 8 warps of 32 keys took 31.6.
#include <cstring>

#include "internal.h"
#include "kv8_host.h"
#include "kv8_sched.cuh"

namespace moe {

namespace {

// Warps per CTA and positions per piece: (8 rows, 16 rows).
constexpr int KA_W8 = 8, KA_W16 = 8;
constexpr int KA_U8 = 32, KA_U16 = 32;
constexpr int KA_ST8 = 2, KA_ST16 = 2;         // pieces in flight per warp
__host__ __device__ constexpr int ka_warps(int R) { return R == 8 ? KA_W8 : KA_W16; }
__host__ __device__ constexpr int ka_u(int R) { return R == 8 ? KA_U8 : KA_U16; }
__host__ __device__ constexpr int ka_stages(int R) { return R == 8 ? KA_ST8 : KA_ST16; }
constexpr int KA_COST = 2;                     // a tile's start, in pieces
__host__ __device__ constexpr int ka_half(int D, int R) { return ka_u(R) * D; }       // bytes of a piece's keys (or values)
__host__ __device__ constexpr int ka_own(int D, int R) { return ka_stages(R) * 2 * ka_half(D, R); }   // a warp's ring
__host__ __device__ constexpr int ka_ps(int D) { return D + 4; }            // floats of a partial row: O, references, normaliser
// shared memory: rings (1024-aligned), a part per warp (the tile that began before its run;
// the tile that goes on after it takes the warp's own ring, which is done by then), the line,
// what the parts belong to, barriers and words
__host__ __device__ constexpr int ka_parts(int D, int R) { return ka_warps(R) * R * ka_ps(D) * 4; }
__host__ __device__ constexpr int ka_wsum(int R) { return R * KV8_MAX_CTAS * 4; }   // weights of a tile's CTAs
__host__ __device__ constexpr int ka_smem(int D, int R, int B) {
  return 1024 + ka_warps(R) * ka_own(D, R) + ka_parts(D, R) + ka_wsum(R) + (B + 2) * 8 +
         ka_warps(R) * (8 + ka_stages(R) * 8 + 2 * 32 + R * 4) + 64;
}
static_assert(ka_smem(128, 16, KV8_MAX_SEQS) <= 232448 && ka_smem(128, 8, KV8_MAX_SEQS) <= 232448,
              "shared memory per CTA exceeds 227 KB");
static_assert(ka_warps(8) * ka_stages(8) <= 32 && ka_warps(16) * ka_stages(16) <= 32, "one lane per barrier");
static_assert(16 * ka_ps(128) * 4 <= ka_own(128, 16) && 16 * ka_ps(64) * 4 <= ka_own(64, 16) &&
                  8 * ka_ps(128) * 4 <= ka_own(128, 8) && 8 * ka_ps(64) * 4 <= ka_own(64, 8),
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
constexpr float KA_LOW = -9.0f;                // 32 positions: 32 * 2^-25 = 2^-11 2^-9

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
// One more part of a tile: the parts that came before.
__device__ __forceinline__ unsigned ticket_add(unsigned* p) {
  unsigned old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}
// An 8x8 fp16 matrix held as rows lane / 4, columns 2 (lane % 4) and + 1, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

}  // namespace

// box: rows of the tensor maps' box, 16 (pages of 16 positions) or 32.
template <int D, int R, int FMT>
__global__ void __launch_bounds__(ka_warps(R) * 32, 1)
    kv8_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ Kv8AttnParams p, int box) {
  constexpr int KA_WARPS = ka_warps(R), KA_THREADS = KA_WARPS * 32, KA_U = ka_u(R), KA_STAGES = ka_stages(R);
  constexpr int HALF = ka_half(D, R), OWN = ka_own(D, R);
  constexpr int NJ = D / 16;          // MMAs of a score tile's contraction
  constexpr int NM = D / 16;          // 16-dim tiles of O^T
  constexpr int NB = R / 8;           // 8-row blocks of queries
  constexpr int NK = KA_U / 16;       // 16-key tiles of a piece
  constexpr int LD = D / 4;           // dims of a key that a lane's quad member holds
  constexpr int VD = D / 8;           // dims of O and V that a lane holds
  constexpr int PS = ka_ps(D);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* heads = reinterpret_cast<float*>(smem + KA_WARPS * OWN);
  float* wsum = heads + ka_parts(D, R) / 4;
  long long* prefix = reinterpret_cast<long long*>(wsum + ka_wsum(R) / 4);
  long long* s_warp = prefix + p.b.n_seqs + 1 + ((p.b.n_seqs + 1) & 1);      // 16-byte aligned
  KaPart* meta = reinterpret_cast<KaPart*>(s_warp + KA_WARPS);             // [warp][began before, goes on]
  uint64_t* bars = reinterpret_cast<uint64_t*>(meta + 2 * KA_WARPS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + KA_WARPS * KA_STAGES);
  int* s_last = const_cast<int*>(abort_flag) + 1;
  float* s_peak = reinterpret_cast<float*>(s_last + 1) + (threadIdx.x >> 5) * R;   // [R] the highest ms + d of a row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g4 = lane >> 2, c4 = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * OWN;
  const uint32_t bar0 = smem_u32(bars) + warp * KA_STAGES * 8;

  if (warp == KA_WARPS - 1) {
    if (lane < KA_WARPS * KA_STAGES) mbar_init(smem_u32(bars) + 8 * lane, 1);
    if (lane == 0) *abort_flag = 0;
    if (lane < 2) tma_prefetch_desc(lane ? &tm_v : &tm_k);
    fence_mbar_init();
  }
  if (tid < 2 * KA_WARPS) meta[tid].b = -1;
  grid_dep_wait();                          // what follows reads and writes what earlier kernels wrote
  Kv8Runs runs;
  runs.total = kv8_line<KA_U, KA_COST, KA_THREADS>(p, prefix, s_warp);
  runs.n = static_cast<int>(min(runs.total, static_cast<long long>(gridDim.x) * KA_WARPS));
  const int cta = blockIdx.x, run = cta * KA_WARPS + warp;
  if (cta * KA_WARPS >= runs.n) return;
  const long long w_beg = run < runs.n ? kv8_run_begin(runs, run) : 0;
  const long long w_end = run < runs.n ? kv8_run_begin(runs, run + 1) : 0;

  // ---- this warp's load cursor: its next piece, and in the first lanes the page of one of the
  // piece's blocks each (first those of the keys, then those of the values)
  const int block = lane % NK, which = lane / NK;
  const bool loader = lane < 2 * NK;
  long long lw = w_beg;
  Kv8Seg ls = {};
  int lu = 0, l_end = 0, pid = -1;
  bool more = w_beg < w_end;
  if (more) {
    ls = kv8_seg<KA_U, KA_COST>(p, prefix, lw, w_end);
    lu = ls.u0;
    l_end = kv8_seg_end(ls, p.tq_shift);
  }
  const Kv8Seg first_seg = ls;
  auto settle = [&] {                 // the cursor's next piece: its segment and its pages
    if (!more) return;
#pragma unroll 1
    while (lu >= ls.u1) {
      lw += ls.len;
      if (lw >= w_end) {
        more = false;
        return;
      }
      kv8_next<KA_U, KA_COST>(ls, p, prefix, lw, w_end);
      lu = ls.u0;
      l_end = kv8_seg_end(ls, p.tq_shift);
    }
    const int pos = lu * KA_U + block * KV8_BLOCK;
    pid = -1;
    if (loader && pos < l_end)
      pid = __ldg(p.b.page_table + static_cast<size_t>(ls.b) * p.b.max_pages + (pos >> p.c.page_shift));
  };
  // Codes that one tile alone reads need no place in L2 (8 x 32768 positions: 31.0 us, 31.9 with the
  // usual policy; which one the codes of several tiles get made no difference).  Pages that
  // sequences share are taken for read once, too.
  const uint64_t pol = p.b.max_new <= (1 << p.tq_shift) ? l2_policy_evict_first() : l2_policy_evict_normal();
  int issued = 0;
  // Issue the cursor's piece into its stage; returns this lane's block scale (the loaders).
  auto issue = [&]() -> float {
    float sc = KA_NO_BLOCK;
    if (!more) return sc;
    const int st = issued % KA_STAGES;
    const int pos = lu * KA_U + block * KV8_BLOCK;
    bool live = loader && pos < l_end;
    if (live && (pid < 0 || pid >= p.c.n_pages)) {
      atomicOr(p.c.err, ERRBIT_BOUNDS);
      live = false;
    }
    size_t row = 0;
    if (live) {
      row = ((static_cast<size_t>(pid) * p.c.hkv + ls.g) << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1));
      sc = __ldg(p.c.scales[which] + row / KV8_BLOCK);     // not looked at before the piece is
    }
    const bool copies = live && (box == KV8_BLOCK || block == 0);   // a box of 32 rows brings both blocks
    const unsigned n = __popc(__ballot_sync(0xffffffffu, copies));
    const uint32_t bar = bar0 + 8 * st;
    if (lane == 0) mbar_arrive_expect_tx(bar, n * box * D);
    __syncwarp();
    if (copies) {
      const uint32_t dst = ring + st * 2 * HALF + which * HALF + block * KV8_BLOCK * D;
      tma_load_2d_hint(dst, which ? &tm_v : &tm_k, bar, 0, static_cast<int>(row), pol);
    }
    ++issued;
    ++lu;
    settle();
    return sc;
  };

  // The query rows of the first segment are on their way before the first codes are.
  uint4 qv[NB][LD / 8];
  const auto fetch_q = [&](const Kv8Seg& g) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = g4 + 8 * b, tok = r / p.G, t0 = g.t << p.tq_shift;
#pragma unroll
      for (int i = 0; i < LD / 8; ++i) qv[b][i] = make_uint4(0, 0, 0, 0);
      if (tok < min(1 << p.tq_shift, g.s.n - t0)) {
        const __nv_bfloat16* src =
            p.q + static_cast<size_t>(g.s.off + t0 + tok) * p.q_stride + (g.g * p.G + r - tok * p.G) * D + LD * c4;
#pragma unroll
        for (int i = 0; i < LD / 8; ++i) qv[b][i] = ldg_nc_v4(src + 8 * i);
      }
    }
  };
  if (more) fetch_q(ls);
  bool fetched = more;
  settle();
  float sc_next[KA_STAGES];
#pragma unroll
  for (int i = 0; i < KA_STAGES; ++i) sc_next[i] = issue();

  int taken = 0;
  bool dead = false;      // a wait gave up: nothing more is loaded or computed
  Kv8Seg sg = first_seg;
#pragma unroll 1
  for (long long w = w_beg; w < w_end;) {
    if (w > w_beg) {
      kv8_next<KA_U, KA_COST>(sg, p, prefix, w, w_end);
      fetched = false;
    }
    w += sg.len;
    if (sg.u1 <= sg.u0) continue;     // the run ends before the tile's first piece
    const int end = kv8_seg_end(sg, p.tq_shift);
    const int tok0 = sg.t << p.tq_shift;
    const int ntok = min(1 << p.tq_shift, sg.s.n - tok0);
    const int nrows = ntok * p.G;
    // ---- query fragments (B: row g4 of each block, dims LD c4 ..), then what this lane needs of
    // the rows whose scores it gets, 8 b + 2 c4 + i
    uint32_t qb[NB][NJ][2];
    if (!fetched) fetch_q(sg);
    float rs[NB][2];                  // factor of the row's scores
    int see[NB][2];                   // positions that the row's token sees
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = g4 + 8 * b;
      const uint4* v = qv[b];
      // (a row without a token has zeros for a query and sees all there is, so that it gets references
      // with the others; with none to see, it would have moved them at every piece)
      const int sees = r < nrows ? sg.s.first + tok0 + r / p.G + 1 : end;
      uint32_t big2 = 0;
#pragma unroll
      for (int i = 0; i < LD / 8; ++i) {
        const uint32_t* x = &v[i].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) big2 = __vmaxu2(big2, x[j] & 0x7FFF7FFFu);
      }
      big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 1));
      big2 = __vmaxu2(big2, __shfl_xor_sync(0xffffffffu, big2, 2));
      const uint32_t big = max(big2 >> 16, big2 & 0xFFFFu);
      // the row's largest magnitude lands in [2^13, 2^14): bf16's 8 bits stay exact in fp16
      // down to 2^-28 of it.  What is not finite makes the whole row NaN.
      const int e = min(max(static_cast<int>(big >> 7) - 127 - 13, KV8_Q_MIN_EXP), KV8_Q_MAX_EXP);
      const float f = big >= 0x7F80u ? NAN : pow2i(-e);
      const float rf = big >= 0x7F80u ? NAN : fminf(pow2i(e) * p.scale_log2, KV8_MAX_FACTOR);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const uint32_t* x = &v[j >> 1].x + (j & 1) * 2;
        qb[b][j][0] = pack2_f16(bf16lo(x[0]) * f, bf16hi(x[0]) * f);
        qb[b][j][1] = pack2_f16(bf16lo(x[1]) * f, bf16hi(x[1]) * f);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        rs[b][i] = __shfl_sync(0xffffffffu, rf, 4 * (2 * c4 + i));
        see[b][i] = __shfl_sync(0xffffffffu, sees, 4 * (2 * c4 + i));
      }
    }
    const int least = sg.s.first + tok0 + 1;       // positions that every row sees
    // references of a row's weights and normaliser; l: this lane's share of the normaliser
    float d[NB][2], ms[NB][2], l[NB][2];
    float o[NB][NM][4];
    float reach = -INFINITY;          // the largest d of the lane's rows; infinite where scores are far or none was seen
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool nan = rs[b][i] != rs[b][i];                 // a row of NaN moves no references
        ms[b][i] = nan ? 0.0f : KV8_NO_REF;
        d[b][i] = nan ? KV8_W_LEAST : 0.0f;
        if (!nan) reach = INFINITY;
        l[b][i] = 0.0f;
        s_peak[8 * b + 2 * c4 + i] = KV8_NO_REF;               // by each lane for itself
      }
#pragma unroll
      for (int i = 0; i < NM; ++i) o[b][i][0] = o[b][i][1] = o[b][i][2] = o[b][i][3] = 0.0f;
    }

#pragma unroll 1
    for (int u = sg.u0; u < sg.u1 && !dead; ++u) {
      const int st = taken % KA_STAGES;
      if (!__all_sync(0xffffffffu, mbar_wait(bar0 + 8 * st, (taken / KA_STAGES) & 1, p.c.err, abort_flag, p.wait_ns))) {
        dead = true;
        break;
      }
      ++taken;
      const uint32_t kb = ring + st * 2 * HALF, vb = kb + HALF;
      const float sc = sc_next[0];
      // ---- scores of the piece's 16-key tiles: x[.][k][2 h + i]: key 16 k + 8 h + g4, row 2 c4 + i
      float x[NB][NK][4], ksc[NK], ve[NK];
      bool live[NK];
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        ksc[k] = __shfl_sync(0xffffffffu, sc, k);
        const float vs = __shfl_sync(0xffffffffu, sc, NK + k);
        live[k] = ksc[k] >= 0.0f;
        ksc[k] = fmaxf(ksc[k], 0.0f);
        ve[k] = static_cast<float>(max(scale_exp(vs), KV8_MIN_EXP));
#pragma unroll
        for (int b = 0; b < NB; ++b) x[b][k][0] = x[b][k][1] = x[b][k][2] = x[b][k][3] = 0.0f;
        if (!live[k]) continue;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const uint4 k0 = lds128(kb + code_off<D>(16 * k + g4, (D / 64) * c4 + i));
          const uint4 k1 = lds128(kb + code_off<D>(16 * k + 8 + g4, (D / 64) * c4 + i));
          const uint32_t *w0 = &k0.x, *w1 = &k1.x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t d0 = kv8_flip<FMT>(w0[j]), d1 = kv8_flip<FMT>(w1[j]);
            const uint32_t a0 = kv8_half2<FMT>(d0, 0), a1 = kv8_half2<FMT>(d1, 0);
            const uint32_t a2 = kv8_half2<FMT>(d0, 1), a3 = kv8_half2<FMT>(d1, 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma_f16_16816(x[b][k], a0, a1, a2, a3, qb[b][4 * i + j][0], qb[b][4 * i + j][1]);
          }
        }
      }
      // ---- s + e - m, masked where a row may not see the whole piece
      const bool masked = u * KA_U + KA_U > least || !live[0] || !live[NK - 1];
      float y[NB][NK][4], least_e = ve[0];
#pragma unroll
      for (int k = 1; k < NK; ++k) least_e = fminf(least_e, ve[k]);
      const auto factor = [&](int b, int k, int i) { return fminf(rs[b][i] * ksc[k], KV8_MAX_FACTOR); };
      const auto hidden = [&](int b, int k, int h, int i) {
        return !live[k] || u * KA_U + 16 * k + 8 * h + g4 >= see[b][i];
      };
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f = factor(b, k, i), add = ve[k] - (ms[b][i] + d[b][i]);
#pragma unroll
            for (int h = 0; h < 2; ++h) y[b][k][2 * h + i] = fmaf(x[b][k][2 * h + i], f, add);
          }
      if (masked) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (hidden(b, k, j >> 1, j & 1)) y[b][k][j] = -INFINITY;
      }
      bool move = reach - least_e > KV8_SUM_TOP;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float mx = fmaxf(y[b][0][i], y[b][0][2 + i]);
#pragma unroll
          for (int k = 1; k < NK; ++k) mx = fmaxf(mx, fmaxf(y[b][k][i], y[b][k][2 + i]));
          // too large for fp16, or too small in all lanes of the row
          const bool low = (__ballot_sync(0xffffffffu, mx >= KA_LOW) & (0x11111111u << c4)) == 0;
          move |= mx > KV8_W_TOP || (low && mx > KV8_W_LOST);
        }
      }
      move = __any_sync(0xffffffffu, move);
      if (move) {
        reach = -INFINITY;
        // the references move to the rows' maxima; what was summed so far follows
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float sv[NK][2], at = ms[b][i], top = -INFINITY;
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                sv[k][h] = hidden(b, k, h, i) ? -INFINITY : kv8_end(x[b][k][2 * h + i] * factor(b, k, i));
                at = fmaxf(at, sv[k][h]);
              }
#pragma unroll
            for (int s = 4; s <= 16; s <<= 1) at = fmaxf(at, __shfl_xor_sync(0xffffffffu, at, s));
#pragma unroll
            for (int k = 0; k < NK; ++k) top = fmaxf(top, fmaxf(sv[k][0], sv[k][1]) - at + ve[k]);
#pragma unroll
            for (int s = 4; s <= 16; s <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            const float was = d[b][i] + (ms[b][i] - at);     // d in units of the new ms
            float& peak = s_peak[8 * b + 2 * c4 + i];
            float to = fmaxf(was, top - KV8_W_FIRST);
            if (kv8_down(top, was, KA_LOW, at, peak)) to = top - KV8_W_FIRST;
            peak = fmaxf(peak, at + to);
            reach = fmaxf(reach, fabsf(at) < KV8_FAR ? to : INFINITY);
            const float corr = ex2(was - to);                // from no reference: 0
            l[b][i] *= ex2(ms[b][i] - at);
            ms[b][i] = at;
            d[b][i] = to;
#pragma unroll
            for (int t = 0; t < NM; ++t) {
              o[b][t][i] *= corr;
              o[b][t][2 + i] *= corr;
            }
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h) y[b][k][2 * h + i] = sv[k][h] - at + (ve[k] - to);
          }
      }
      // the normaliser's terms by themselves, where the weights do not give them
      const bool apart = move && __any_sync(0xffffffffu, reach - least_e > KV8_SUM_TOP);
      if (apart) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) l[b][j & 1] += ex2(y[b][k][j] + (d[b][j & 1] - ve[k]));
      }
      uint32_t pb[NB][NK][2];         // weights as B: keys 16 k + 8 h + 2 c4 and + 1 of row g4
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float sum[2] = {0.0f, 0.0f};    // of this piece, as if d were 0
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          float w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = ex2(y[b][k][j]);
          const float inv = pow2i(-static_cast<int>(ve[k]));
          sum[0] = fmaf(w[0] + w[2], inv, sum[0]);
          sum[1] = fmaf(w[1] + w[3], inv, sum[1]);
          pb[b][k][0] = transpose8x8(pack2_f16(w[0], w[1]));
          pb[b][k][1] = transpose8x8(pack2_f16(w[2], w[3]));
        }
        if (!apart) {
          l[b][0] = fmaf(sum[0], ex2(d[b][0]), l[b][0]);
          l[b][1] = fmaf(sum[1], ex2(d[b][1]), l[b][1]);
        }
      }
      // ---- O^T += V^T w, 16 keys a step; rows past the tile's end are not looked at
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        if (!live[k]) continue;
        const int r = 16 * k + 2 * c4;
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
        const int base = u * KA_U + 16 * k;
        if (base + 16 > end) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (base + 2 * c4 + (i & 1) + (i >> 1) * 8 >= end)
#pragma unroll
              for (int j = 0; j < W; ++j) rw[i][j] = 0;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const uint32_t lo01 = kv8_flip<FMT>(__byte_perm(rw[0][j], rw[1][j], 0x5140));
          const uint32_t hi01 = kv8_flip<FMT>(__byte_perm(rw[0][j], rw[1][j], 0x7362));
          const uint32_t lo23 = kv8_flip<FMT>(__byte_perm(rw[2][j], rw[3][j], 0x5140));
          const uint32_t hi23 = kv8_flip<FMT>(__byte_perm(rw[2][j], rw[3][j], 0x7362));
          // tile 2 j + t: dims VD g4 + 4 j + 2 t (rows g4) and + 1 (rows g4 + 8)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t w01 = t ? hi01 : lo01, w23 = t ? hi23 : lo23;
            const uint32_t a0 = kv8_half2<FMT>(w01, 0), a1 = kv8_half2<FMT>(w01, 1);
            const uint32_t a2 = kv8_half2<FMT>(w23, 0), a3 = kv8_half2<FMT>(w23, 1);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma_f16_16816(o[b][2 * j + t], a0, a1, a2, a3, pb[b][k][0], pb[b][k][1]);
          }
        }
      }
      // the stage is free once every lane has read it
      __syncwarp();
#pragma unroll
      for (int i = 0; i + 1 < KA_STAGES; ++i) sc_next[i] = sc_next[i + 1];
      sc_next[KA_STAGES - 1] = issue();
    }

    // ---- the tile's rows: out if the whole tile lies in this run, else a part for the CTA.
    // This lane has dims VD g4 .. of rows 8 b + 2 c4 + i, two per 16-dim tile.
    const bool whole = sg.u0 == 0 && sg.u1 == sg.units;
    if (!whole && sg.u0 == 0) __syncwarp();   // the part goes into the ring: every lane has read its last piece
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[b][i];
#pragma unroll
        for (int s = 4; s <= 16; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        const int r = 8 * b + 2 * c4 + i;
        if (whole) {
          if (r < nrows) {
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;   // a row that saw no key: zeros
            const float unit = ex2(d[b][i]);                     // of the weights, in the normaliser's
            const int tok = r / p.G, hh = r - tok * p.G;
            __nv_bfloat16* dst =
                p.out + (static_cast<size_t>(sg.s.off + tok0 + tok) * p.hq + sg.g * p.G + hh) * D + VD * g4;
#pragma unroll
            for (int t = 0; t < NM; t += 4) {
              uint32_t v[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                v[k] = pack_bf16x2(__float_as_uint(o[b][t + k][i] * inv * unit),
                                   __float_as_uint(o[b][t + k][2 + i] * inv * unit));
              *reinterpret_cast<uint4*>(dst + 2 * t) = make_uint4(v[0], v[1], v[2], v[3]);
            }
          }
        } else {
          float* row = (sg.u0 ? heads + warp * R * PS
                              : reinterpret_cast<float*>(smem + warp * OWN)) + r * PS;
          if (g4 == 0) *reinterpret_cast<float4*>(row + D) = make_float4(ms[b][i], d[b][i], sum, 0.0f);
#pragma unroll
          for (int t = 0; t < NM; t += 2)
            *reinterpret_cast<float4*>(row + VD * g4 + 2 * t) =
                make_float4(o[b][t][i], o[b][t][2 + i], o[b][t + 1][i], o[b][t + 1][2 + i]);
        }
      }
    if (!whole) {
      const int2 own = kv8_owners<KA_COST>(sg, w - sg.len, runs);
      if (lane == 0) meta[2 * warp + (sg.u0 == 0)] = KaPart{sg.b, sg.g, sg.t, sg.s.off, sg.s.n, own.x, own.y, 0};
    }
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
#pragma unroll 1
  for (int i0 = -1; i0 < KA_WARPS; ++i0) {
    const KaPart pt = i0 < 0 ? meta[0] : meta[2 * i0 + 1];
    if (pt.b < 0) continue;
    const int last = min(pt.r_last - cta * KA_WARPS, KA_WARPS - 1);   // the tile's last warp here
    const int c_first = pt.r_first / KA_WARPS, c_last = pt.r_last / KA_WARPS;
    const auto part = [&](int i) {           // i0: the tail (or nothing, for -1), above: heads
      return (i == i0 ? reinterpret_cast<const float*>(smem + i * OWN) : heads + i * R * PS) + row * PS;
    };
    const int i1 = max(i0, 0);
    float M = KV8_NO_REF, top = -INFINITY, L = 0.0f, O[8] = {0, 0, 0, 0, 0, 0, 0, 0};   // references ms and d
    if (tid < ACT) {
      // unrolled over all warps, so that the loads do not wait for one another
      float mw[KA_WARPS], dw[KA_WARPS], lw2[KA_WARPS];
#pragma unroll
      for (int i = 0; i < KA_WARPS; ++i) {
        mw[i] = KV8_NO_REF;
        dw[i] = lw2[i] = 0.0f;
        if (i >= i1 && i <= last) {
          const float4 v = *reinterpret_cast<const float4*>(part(i) + D);
          mw[i] = v.x;
          dw[i] = v.y;
          lw2[i] = v.z;
        }
        M = fmaxf(M, mw[i]);
      }
#pragma unroll
      for (int i = 0; i < KA_WARPS; ++i)
        if (i >= i1 && i <= last) top = fmaxf(top, mw[i] - M + dw[i]);
#pragma unroll
      for (int i = 0; i < KA_WARPS; ++i) {
        if (i < i1 || i > last) continue;
        const float4 v0 = *reinterpret_cast<const float4*>(part(i) + d0), v1 = *reinterpret_cast<const float4*>(part(i) + d0 + 4);
        const float f = ex2(mw[i] - M + dw[i] - top);
        L = fmaf(ex2(mw[i] - M), lw2[i], L);
        O[0] = fmaf(f, v0.x, O[0]), O[1] = fmaf(f, v0.y, O[1]), O[2] = fmaf(f, v0.z, O[2]), O[3] = fmaf(f, v0.w, O[3]);
        O[4] = fmaf(f, v1.x, O[4]), O[5] = fmaf(f, v1.y, O[5]), O[6] = fmaf(f, v1.z, O[6]), O[7] = fmaf(f, v1.w, O[7]);
      }
    }
    bool write = c_first == c_last;
    if (!write) {
      const auto slot = [&](int c) { return p.part + ((static_cast<size_t>(c) * 2 + (c == c_first)) * R + row) * PS; };
      if (tid < ACT) {
        float* dst = slot(cta);
        *reinterpret_cast<float4*>(dst + d0) = make_float4(O[0], O[1], O[2], O[3]);
        *reinterpret_cast<float4*>(dst + d0 + 4) = make_float4(O[4], O[5], O[6], O[7]);
        if (d0 == 0) *reinterpret_cast<float4*>(dst + D) = make_float4(M, top, L, 0.0f);
      }
      __syncthreads();
      const int ns = c_last - c_first + 1;
      if (tid == 0) {
        // release after the barrier, so the whole CTA's sums come before the ticket; acquire for
        // the CTA that adds them up
        const bool all = ticket_add(p.tickets + c_first) == static_cast<unsigned>(ns) - 1u;
        if (all) p.tickets[c_first] = 0u;    // every part has arrived: ready for the next call
        *s_last = all;
      }
      __syncthreads();
      write = *s_last != 0;
      if (write) {
        float* fs = wsum;                    // [R][ns] weights of the CTAs' sums, in the order of the line
        L = 0.0f;
        if (tid < ACT) {
          const int j0 = tid % TPR;
          constexpr int PER = (KV8_MAX_CTAS + TPR - 1) / TPR;
          float ml[PER], dl[PER], ll[PER];
          M = KV8_NO_REF;
          top = -INFINITY;
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int i = j0 + k * TPR;
            ml[k] = KV8_NO_REF;
            dl[k] = -INFINITY;
            ll[k] = 0.0f;
            if (i < ns) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(slot(c_first + i) + D));
              ml[k] = v.x;
              dl[k] = v.y;
              ll[k] = v.z;
            }
          }
#pragma unroll
          for (int k = 0; k < PER; ++k) M = fmaxf(M, ml[k]);
#pragma unroll
          for (int s = TPR / 2; s >= 1; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            L = fmaf(ex2(ml[k] - M), ll[k], L);
            dl[k] += ml[k] - M;
            top = fmaxf(top, dl[k]);
          }
#pragma unroll
          for (int s = TPR / 2; s >= 1; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
#pragma unroll
          for (int k = 0; k < PER; ++k) {
            const int i = j0 + k * TPR;
            if (i < ns) fs[row * ns + i] = ex2(dl[k] - top);
          }
#pragma unroll
          for (int s = TPR / 2; s >= 1; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
        }
        __syncthreads();
        if (tid < ACT) {
#pragma unroll
          for (int k = 0; k < 8; ++k) O[k] = 0.0f;
#pragma unroll 8
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
      const float unit = ex2(top);
      const int tok = row / p.G, hh = row - tok * p.G;
      uint4 r;
      r.x = pack_bf16x2(__float_as_uint(O[0] * inv * unit), __float_as_uint(O[1] * inv * unit));
      r.y = pack_bf16x2(__float_as_uint(O[2] * inv * unit), __float_as_uint(O[3] * inv * unit));
      r.z = pack_bf16x2(__float_as_uint(O[4] * inv * unit), __float_as_uint(O[5] * inv * unit));
      r.w = pack_bf16x2(__float_as_uint(O[6] * inv * unit), __float_as_uint(O[7] * inv * unit));
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

// Query rows of a tile, or 0 for the prompt kernel.  Up to 32 rows go through the decode
// kernel in tiles of 16, each of which reads the codes again, mostly from L2: 4 new tokens of 8
// query heads each, two tiles, took 28 us that way over 16 sequences of 8 thousand positions and
// 18 over one, and 36 and 25 in one block of 128 rows, three quarters empty.  With 64 rows, four
// tiles, it was 53 and 17 against 36 and 25.  A tile holds a power of two of tokens, so that
// other numbers of query heads make three tiles of up to 32 rows (5 heads, 6 tokens: 2 a tile);
// those were not measured.
int ka_rows(int G, int max_new) {
  const long long n = static_cast<long long>(G) * max_new;
  return n <= 8 ? 8 : n <= 32 ? 16 : 0;
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
  return launch_pdl(k, dim3(grid), dim3(ka_warps(R) * 32), ka_smem(D, R, p.b.n_seqs), s, tk, tv, p, box);
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
  const int box = cache->page_size >= ka_u(R) ? ka_u(R) : KV8_BLOCK;
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
