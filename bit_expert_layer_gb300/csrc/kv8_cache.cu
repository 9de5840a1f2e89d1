// kv8_cache.cu -- the 8-bit key/value cache's write and read back, and rotary positions, with or
// without norms of the heads.
// All are bound by memory: each reads its rows once and writes them once.  Measured on 2
// key/value and 16 query heads of 128: the write of 16 thousand tokens (int8, 23 MB) 5.9 us
// (3.5 at the copy rate), 60 thousand rows read back (e4m3, 92 MB) 15.1 us (13.8), 16384 tokens
// rotated (151 MB) 28.0 us (22.6), normed and rotated 29.6 us.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "kv8.cuh"
#include "kv8_host.h"

namespace moe {

namespace {

constexpr int KC_WARPS = 8;
constexpr float BF16_MAX = 3.3895313892515355e38f;

struct Kv8RowsParams {
  Kv8Cache c;
  Kv8Batch b;
  const __nv_bfloat16* in[2];   // append: k, v
  __nv_bfloat16* out[2];        // gather: k, v
  long long stride[2];          // append: elements between rows
  int units;
};

// What one warp works on: a 16-position block of one sequence and head, keys or values.
struct Kv8Block {
  Kv8Seq s;
  int g, kv;
  int pos0;        // first position of the block
  bool live;
  size_t at;       // code row (of head_size bytes) of pos0 in the cache; / 16 = its scale
};

__device__ __forceinline__ Kv8Block kv8_block(const Kv8RowsParams& p) {
  grid_dep_wait();
  Kv8Block k;
  k.live = false;
  // consecutive warps take the keys and values of all heads of a unit, then the next unit
  const long long id = static_cast<long long>(blockIdx.x) * KC_WARPS + (threadIdx.x >> 5);
  k.kv = static_cast<int>(id & 1);
  const long long r = id >> 1;
  const int u = static_cast<int>(r / p.c.hkv);
  k.g = static_cast<int>(r - static_cast<long long>(u) * p.c.hkv);
  if (u >= p.units) return k;
  const int b = kv8_unit_seq(p.b, u);
  k.s = kv8_seq(p.b, p.c.page_shift, b);
  const bool report = lane_id() == 0;
  if (k.s.bad && report) atomicOr(p.c.err, ERRBIT_BOUNDS);
  const int j = u - (k.s.off / KV8_BLOCK + 2 * b);
  if (k.s.n <= 0) return k;
  if (k.s.first < 0 && report) atomicOr(p.c.err, ERRBIT_BOUNDS);   // more new tokens than positions
  const int blk = max(k.s.first, 0) / KV8_BLOCK + j;
  k.pos0 = blk * KV8_BLOCK;
  if (j < 0 || k.pos0 >= k.s.first + k.s.n) return k;
  const int page = __ldg(p.b.page_table + static_cast<size_t>(b) * p.b.max_pages + (k.pos0 >> p.c.page_shift));
  if (page < 0 || page >= p.c.n_pages) {
    if (report) atomicOr(p.c.err, ERRBIT_BOUNDS);
    return k;
  }
  k.at = ((static_cast<size_t>(page) * p.c.hkv + k.g) << p.c.page_shift) + (k.pos0 & ((1 << p.c.page_shift) - 1));
  k.live = true;
  return k;
}

}  // namespace

// Cache write.  One warp per (16-position block, head, keys or values): a lane holds 8
// elements of every second (D = 128) or fourth (D = 64) row, so a row moves as 16-byte
// loads and 8-byte stores, and the block's largest magnitude is a butterfly of bf16 bits.
// Since a block belongs to one warp, its scale and its older codes change with no atomics.
// (What is not finite is looked for only where the maximum says that it is there: with the test
// on every element the kernel took 127 registers and 9.5 us on the case above.)
template <int D, int FMT>
__global__ void __launch_bounds__(KC_WARPS * 32) kv8_append_kernel(const __grid_constant__ Kv8RowsParams p) {
  constexpr int LPR = D / 8;             // lanes per row
  constexpr int RPI = 32 / LPR;          // rows per step
  constexpr int NI = KV8_BLOCK / RPI;
  const Kv8Block k = kv8_block(p);
  if (!k.live) return;
  const int lane = lane_id(), r0 = lane / LPR, d0 = (lane % LPR) * 8;
  uint8_t* codes = p.c.codes[k.kv] + k.at * D + d0;
  float* scale = p.c.scales[k.kv] + k.at / KV8_BLOCK;
  const int lo = max(k.s.first, 0) - k.pos0, hi = k.s.first + k.s.n - k.pos0;   // new rows of the block: lo .. hi - 1
  const bool held = lo > 0;                                          // rows 0 .. lo - 1 hold earlier positions
  const __nv_bfloat16* src = p.in[k.kv] + static_cast<size_t>(k.g) * D + d0;

  uint4 x[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = r0 + i * RPI;
    x[i] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi)
      x[i] = ldg_nc_v4(src + static_cast<size_t>(k.s.off + k.pos0 + r - k.s.first) * p.stride[k.kv]);
  }
  float s_old = 0.0f;
  if (held) s_old = *scale;
  uint32_t big2 = 0;                     // largest magnitudes, as pairs of bf16 bits
#pragma unroll
  for (int i = 0; i < NI; ++i)
    big2 = __vmaxu2(__vmaxu2(big2, __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu)),
                    __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
  uint32_t amax = __reduce_max_sync(0xffffffffu, max(big2 & 0xFFFFu, big2 >> 16));
  if (amax >= 0x7F80u) {
    // something is not finite: it does not count, and a NaN becomes zero
    if (lane == 0) atomicOr(p.c.err, ERRBIT_NONFINITE);
    amax = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) amax = max(amax, lo);
        if (hi < 0x7F80u) amax = max(amax, hi);
        if (lo > 0x7F80u) w[j] &= 0xFFFF0000u;
        if (hi > 0x7F80u) w[j] &= 0x0000FFFFu;
      }
      x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    amax = __reduce_max_sync(0xffffffffu, amax);
  }
  int e = kv8_exp_of<FMT>(amax);
  if (held) {
    const int e_old = max(scale_exp(s_old), KV8_MIN_EXP);
    if (e > e_old) {
      // the earlier rows' codes, rounded again to the larger scale
      const float f = pow2i(max(e_old - e, -126));
#pragma unroll 1
      for (int r = r0; r < lo; r += RPI) {
        const uint2 c = *reinterpret_cast<const uint2*>(codes + r * D);
        uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t v = kv8_flip<FMT>(w[j]);
          const float2 a = half2_floats(kv8_half2<FMT>(v, 0)), b = half2_floats(kv8_half2<FMT>(v, 1));
          w[j] = kv8_encode4<FMT>(a.x * f, a.y * f, b.x * f, b.y * f);
        }
        *reinterpret_cast<uint2*>(codes + r * D) = make_uint2(w[0], w[1]);
      }
    } else {
      e = e_old;
    }
  }
  const float inv = pow2i(-e);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = r0 + i * RPI;
    if (r < lo || r >= hi) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint2 c;
    c.x = kv8_encode4<FMT>(bf16lo(w[0]) * inv, bf16hi(w[0]) * inv, bf16lo(w[1]) * inv, bf16hi(w[1]) * inv);
    c.y = kv8_encode4<FMT>(bf16lo(w[2]) * inv, bf16hi(w[2]) * inv, bf16lo(w[3]) * inv, bf16hi(w[3]) * inv);
    *reinterpret_cast<uint2*>(codes + r * D) = c;
  }
  if (lane == 0) *scale = pow2i(e);
}

// Read back, the same shape of work: 8-byte loads of codes, 16-byte stores of bf16.  A code
// has at most 8 significant bits, so code * scale is exact in bf16; only 256 * 2^120, the
// e4m3 number next to bf16's largest ones, is past its range and comes back as the largest.
template <int D, int FMT>
__global__ void __launch_bounds__(KC_WARPS * 32) kv8_gather_kernel(const __grid_constant__ Kv8RowsParams p) {
  constexpr int LPR = D / 8;
  constexpr int RPI = 32 / LPR;
  constexpr int NI = KV8_BLOCK / RPI;
  const Kv8Block k = kv8_block(p);
  if (!k.live) return;
  const int lane = lane_id(), r0 = lane / LPR, d0 = (lane % LPR) * 8;
  const uint8_t* codes = p.c.codes[k.kv] + k.at * D + d0;
  const int lo = max(k.s.first, 0) - k.pos0, hi = k.s.first + k.s.n - k.pos0;
  uint2 c[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = r0 + i * RPI;
    c[i] = make_uint2(0, 0);
    if (r >= lo && r < hi) c[i] = __ldg(reinterpret_cast<const uint2*>(codes + r * D));
  }
  const float s = __ldg(p.c.scales[k.kv] + k.at / KV8_BLOCK);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int r = r0 + i * RPI;
    if (r < lo || r >= hi) continue;
    const uint32_t w[2] = {kv8_flip<FMT>(c[i].x), kv8_flip<FMT>(c[i].y)};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = half2_floats(kv8_half2<FMT>(w[j >> 1], j & 1));
      const float x = fminf(fmaxf(f.x * s, -BF16_MAX), BF16_MAX), y = fminf(fmaxf(f.y * s, -BF16_MAX), BF16_MAX);
      const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
      o[j] = *reinterpret_cast<const uint32_t*>(&v);
    }
    const size_t t = static_cast<size_t>(k.s.off + k.pos0 + r - k.s.first);
    *reinterpret_cast<uint4*>(p.out[k.kv] + (t * p.c.hkv + k.g) * D + d0) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// ============================================================================ rotary positions
namespace {

constexpr int RP_THREADS = 256;

struct RopeParams {
  const __nv_bfloat16* in[2];    // q, k
  __nv_bfloat16* out[2];
  long long in_stride[2], out_stride[2];
  int heads[2];
  const int* pos;
  int T, n_axes, half, tokens;   // tokens per CTA, at most 4
  uint32_t inv_heads;            // th / heads = th inv_heads >> 21 for th < 4 heads, heads <= 512 (norms: 32 and 128 steps)
  uint64_t turn[GQA_ROPE_MAX_PAIRS];
  uint8_t axis[GQA_ROPE_MAX_PAIRS];
  const void* weight[2];         // norms: of the q heads, the k heads (null: ones)
  int weight_f32;
  float eps, offset;
};

}  // namespace

// Rotary positions.  pos * turn is exact modulo one turn in 64-bit arithmetic, its top bits
// as a signed fraction of a half turn go to sincospif.  A CTA computes the sines of its
// tokens once into shared memory and turns all heads with them.  Its work items are two
// 16-byte chunks of a head: chunk i with chunk i + half / 8 of the rotated part, or two
// chunks of the part that passes through.
template <int D>
__global__ void __launch_bounds__(RP_THREADS) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float s_cs[];        // [tokens][half] cosines, then sines
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
  float* s_cos = s_cs;
  float* s_sin = s_cs + p.tokens * p.half;
  constexpr int IPH = D / 16;            // items per head
  constexpr int NB = 3;                  // items of a thread in flight: 4 tokens of 18 heads of 128
  const int rot_items = p.half / 8, nh = p.heads[0] + p.heads[1], n = nt * nh * IPH;
  struct Item {
    const __nv_bfloat16* src;
    __nv_bfloat16* dst;
    int ca, cb, at;                      // its chunks' first elements; of its sines, or -1
  };
  const auto item = [&](int i) {
    Item r;
    const int part = i % IPH, th = i / IPH;
    const int t = static_cast<int>((static_cast<uint32_t>(th) * p.inv_heads) >> 21), hh = th - t * nh;
    const int which = hh >= p.heads[0];
    const int h = which ? hh - p.heads[0] : hh;
    r.src = p.in[which] + static_cast<size_t>(t0 + t) * p.in_stride[which] + h * D;
    r.dst = p.out[which] + static_cast<size_t>(t0 + t) * p.out_stride[which] + h * D;
    const bool rot = part < rot_items;
    r.ca = rot ? part * 8 : 2 * p.half + (part - rot_items) * 16;
    r.cb = rot ? r.ca + p.half : r.ca + 8;
    r.at = rot ? t * p.half + part * 8 : -1;
    return r;
  };
  uint4 a[NB], b[NB];
  const auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = i0 + k * RP_THREADS;
      if (i < n) {
        const Item r = item(i);
        a[k] = *reinterpret_cast<const uint4*>(r.src + r.ca);
        b[k] = *reinterpret_cast<const uint4*>(r.src + r.cb);
      }
    }
  };
  grid_dep_wait();
  load(threadIdx.x);                     // on their way while the sines are computed
  for (int i = threadIdx.x; i < nt * p.half; i += RP_THREADS) {
    const int t = i / p.half, j = i - t * p.half;
    const long long pos = __ldg(p.pos + static_cast<size_t>(p.axis[j]) * p.T + t0 + t);
    const long long frac = static_cast<long long>(static_cast<unsigned long long>(pos) * p.turn[j]);
    float s, c;
    sincospif(static_cast<float>(frac) * 1.0842021724855044e-19f /* 2^-63 */, &s, &c);
    s_cos[i] = c;
    s_sin[i] = s;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < n; i0 += NB * RP_THREADS) {
    if (i0 != threadIdx.x) load(i0);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = i0 + k * RP_THREADS;
      if (i >= n) break;
      const Item r = item(i);
      if (r.at >= 0) {
        uint32_t *wa = &a[k].x, *wb = &b[k].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 c = *reinterpret_cast<const float2*>(s_cos + r.at + 2 * j);
          const float2 s = *reinterpret_cast<const float2*>(s_sin + r.at + 2 * j);
          const float a0 = bf16lo(wa[j]), a1 = bf16hi(wa[j]), b0 = bf16lo(wb[j]), b1 = bf16hi(wb[j]);
          wa[j] = pack_bf16x2(__float_as_uint(a0 * c.x - b0 * s.x), __float_as_uint(a1 * c.y - b1 * s.y));
          wb[j] = pack_bf16x2(__float_as_uint(b0 * c.x + a0 * s.x), __float_as_uint(b1 * c.y + a1 * s.y));
        }
      }
      *reinterpret_cast<uint4*>(r.dst + r.ca) = a[k];
      *reinterpret_cast<uint4*>(r.dst + r.cb) = b[k];
    }
  }
}

// ============================================================================ norms and rotary positions
namespace {

constexpr int NR_TOKENS = 32;              // tokens of a CTA at most
constexpr int NR_CTAS = 4;                 // resident CTAs per SM (64 registers)

// Sums of squares between these need no care: none of their terms that matter left fp32's range.
constexpr float NORM_LEAST = 0x1p-80f;
constexpr float NORM_LEAST_EPS = 0x1p-60f;       // beside it, smaller sums do not matter

// A head whose squares leave fp32 (magnitudes over 2^60 or under 2^-45): its root mean square in
// 64 bits, by the head's IPH threads.  Returns a power of two next to its reciprocal and the rest
// of it, so that neither product leaves fp32.  Infinities make the others zeros and themselves NaN,
// as the formula does.  (By value: a thread's elements stay in registers on the ordinary way.)
template <int IPH>
__device__ __noinline__ float2 norm_far(uint4 a, uint4 b, uint32_t mask, float eps) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  double sum = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const double lo = bf16lo(w[j]), hi = bf16hi(w[j]);
    sum += lo * lo + hi * hi;
  }
#pragma unroll
  for (int m = IPH / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(mask, sum, m);
  const double root = sqrt(sum / (16 * IPH) + eps);
  if (root == 0.0) return make_float2(1.0f, 0.0f);       // zeros with eps 0 stay zeros
  const int e = isfinite(root) ? min(max(ilogb(root), -126), 126) : 0;
  return make_float2(pow2i(-e), static_cast<float>(1.0 / (root * pow2i(-e))));
}

}  // namespace

// Norms of the heads with the rotary positions.  A CTA has some tokens and computes their sines once.
// D / 16 neighbouring lanes share a head (two 16-byte chunks each, as in rope_kernel) and add
// their squares by shuffles, so a step of a warp is 512 / D heads of q or of k of one token, and a
// lane keeps its place in the head from step to step.  Arithmetic goes two elements at a time;
// sines, negated sines and weights (as factors) lie in shared memory with the halves of the
// 8-element chunks apart, so that neighbours' 16-byte loads lie side by side.
// Bound: memory (151 MB for 16384 tokens of 18 heads of 128: 22.5 us at a copy's rate); measured 29.6 us,
// 5.1 TB/s, some 250 instructions a step at 0.7 a cycle and scheduler.  On the way there: 94.7 us with
// a head's elements in local memory (their address went to the rare function), 37 to 39 with scalar
// arithmetic and four tokens a CTA, whatever the registers; a warp per token, steps prefetched by
// asynchronous copies, 31.6, but 5 us where this takes 2.5 (256 tokens).
template <int D>
__global__ void __launch_bounds__(RP_THREADS, NR_CTAS) norm_rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) float s_cs[];          // [tokens][half] cosines, sines, negated sines, then [2][D] weights
  __shared__ uint64_t s_turn[GQA_ROPE_MAX_PAIRS];
  __shared__ const int* s_pos[GQA_ROPE_MAX_PAIRS];
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0), half = p.half;
  const int all = p.tokens * half;
  float* s_w = s_cs + 3 * all;
  constexpr int IPH = D / 16, NG = 32 / IPH, WARPS = RP_THREADS / 32;      // lanes of a head, heads of a step
  constexpr int NB = 2;                  // steps of a warp in flight
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31, part = lane % IPH, grp = lane / IPH;
  const bool rot = part < half / 8;
  const int ca = rot ? part * 8 : 2 * half + (part - half / 8) * 16, gap = rot ? half : 8, own = grp * D + ca;
  const int nq = (p.heads[0] + NG - 1) / NG, per = nq + (p.heads[1] + NG - 1) / NG, n = nt * per;
  struct Step {
    const __nv_bfloat16* src;            // the step's first head
    __nv_bfloat16* dst;
    const float *w, *cs;                 // its weights, its token's sines
    bool live;                           // the lane's head exists
  };
  const auto step = [&](int i) {
    Step r;
    const int t = (static_cast<uint32_t>(i) * p.inv_heads) >> 21, st = i - t * per;
    if (st < nq) {
      r.src = p.in[0] + (t0 + t) * p.in_stride[0] + st * NG * D;
      r.dst = p.out[0] + (t0 + t) * p.out_stride[0] + st * NG * D;
      r.live = st * NG + grp < p.heads[0];
      r.w = s_w;
    } else {
      r.src = p.in[1] + (t0 + t) * p.in_stride[1] + (st - nq) * NG * D;
      r.dst = p.out[1] + (t0 + t) * p.out_stride[1] + (st - nq) * NG * D;
      r.live = (st - nq) * NG + grp < p.heads[1];
      r.w = s_w + D;
    }
    r.cs = s_cs + t * half;
    return r;
  };
  uint4 a[NB], b[NB];
  Step at[NB];
  const auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      a[k] = b[k] = make_uint4(0, 0, 0, 0);
      const int i = i0 + k * WARPS;
      if (i >= n) break;
      at[k] = step(i);
      if (at[k].live) {
        a[k] = *reinterpret_cast<const uint4*>(at[k].src + own);
        b[k] = *reinterpret_cast<const uint4*>(at[k].src + own + gap);
      }
    }
  };
  if (threadIdx.x < half) {
    s_turn[threadIdx.x] = p.turn[threadIdx.x];
    s_pos[threadIdx.x] = p.pos + static_cast<size_t>(p.axis[threadIdx.x]) * p.T + t0;
  }
  grid_dep_wait();
  load(warp);                            // on their way while the sines are computed
  __syncthreads();
  const int rows = RP_THREADS / half, row = threadIdx.x / half, j = threadIdx.x - row * half;
  if (row < rows) {
    float* to = s_cs + (j >> 2 & 1) * (half / 2) + (j >> 3) * 4 + (j & 3);
    const uint64_t turn = s_turn[j];
    const int* pos = s_pos[j];
    for (int t = row; t < nt; t += rows) {
      const long long frac = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(__ldg(pos + t))) * turn);
      float s, c;
      sincospif(static_cast<float>(frac) * 1.0842021724855044e-19f /* 2^-63 */, &s, &c);
      to[t * half] = c;
      to[t * half + all] = s;
      to[t * half + 2 * all] = -s;
    }
  }
  for (int i = threadIdx.x; i < 2 * D; i += RP_THREADS) {
    const int which = i / D, e = i % D;
    const void* w = which ? p.weight[1] : p.weight[0];
    float v = 1.0f;
    if (w) v = (p.weight_f32 ? __ldg(static_cast<const float*>(w) + e) : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(w) + e))) + p.offset;
    s_w[which * D + (e >> 2 & 1) * (D / 2) + (e >> 3) * 4 + (e & 3)] = v;
  }
  __syncthreads();
#pragma unroll 1
  for (int i0 = warp; i0 < n; i0 += NB * WARPS) {
    if (i0 != warp) load(i0);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      if (i0 + k * WARPS >= n) break;
      const uint32_t w[8] = {a[k].x, a[k].y, a[k].z, a[k].w, b[k].x, b[k].y, b[k].z, b[k].w};
      uint64_t x[8], sum2[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = f32x2(bf16lo(w[j]), bf16hi(w[j]));
        sum2[j & 1] = fma2(x[j], x[j], sum2[j & 1]);
      }
      const float2 both = f32x2_get(add2(sum2[0], sum2[1]));
      float sum = both.x + both.y;
#pragma unroll
      for (int m = IPH / 2; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
      float f;
      if (sum <= 0x1p120f && (sum >= NORM_LEAST || p.eps >= NORM_LEAST_EPS)) {
        f = rsqrtf(fmaf(sum, 1.0f / D, p.eps));
      } else {
        // by the head's lanes: other heads of the step may be ordinary ones
        const float2 r2 = norm_far<IPH>(a[k], b[k], ((1u << IPH) - 1) << (grp * IPH), p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = mul2(x[j], f32x2(r2.x, r2.x));
        f = r2.y;
      }
      const float *wt = at[k].w + ca / 2, *cs = at[k].cs + part * 4;
      const uint64_t f2 = f32x2(f, f);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const ulonglong2 wa = *reinterpret_cast<const ulonglong2*>(wt + q * (D / 2));
        const ulonglong2 wb = *reinterpret_cast<const ulonglong2*>(wt + gap / 2 + q * (D / 2));
        const uint64_t u[2] = {wa.x, wa.y}, v[2] = {wb.x, wb.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          x[2 * q + j] = mul2(mul2(x[2 * q + j], f2), u[j]);
          x[4 + 2 * q + j] = mul2(mul2(x[4 + 2 * q + j], f2), v[j]);
        }
        if (rot) {
          const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(cs + q * (half / 2));
          const ulonglong2 s2 = *reinterpret_cast<const ulonglong2*>(cs + all + q * (half / 2));
          const ulonglong2 n2 = *reinterpret_cast<const ulonglong2*>(cs + 2 * all + q * (half / 2));
          const uint64_t c[2] = {c2.x, c2.y}, s[2] = {s2.x, s2.y}, ns[2] = {n2.x, n2.y};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint64_t a0 = x[2 * q + j], b0 = x[4 + 2 * q + j];
            x[2 * q + j] = fma2(b0, ns[j], mul2(a0, c[j]));
            x[4 + 2 * q + j] = fma2(a0, s[j], mul2(b0, c[j]));
          }
        }
      }
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 y = f32x2_get(x[j]);
        o[j] = pack_bf16x2(__float_as_uint(y.x), __float_as_uint(y.y));
      }
      if (at[k].live) {
        *reinterpret_cast<uint4*>(at[k].dst + own) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(at[k].dst + own + gap) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
  }
}

}  // namespace moe

// ============================================================================ C ABI
namespace moe {

bool kv8_cache_ok(const gqa_kv8_cache_t* c, moe_status_t* st) {
  *st = MOE_ERR_INVALID_ARG;
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !c->error) return false;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 64) return false;
  if (c->page_size < KV8_BLOCK || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return false;
  if (c->head_size != 64 && c->head_size != 128) return false;
  if (c->format != GQA_KV8_E4M3 && c->format != GQA_KV8_INT8) return false;
  if (static_cast<long long>(c->n_pages) * c->n_kv_heads * c->page_size > 0x7FFFFFFFll) return false;
  *st = MOE_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(c->k_codes) | reinterpret_cast<uintptr_t>(c->v_codes)) & 15u) return false;
  if ((reinterpret_cast<uintptr_t>(c->k_scales) | reinterpret_cast<uintptr_t>(c->v_scales) |
       reinterpret_cast<uintptr_t>(c->error)) & 3u)
    return false;
  *st = MOE_OK;
  return true;
}

bool kv8_batch_ok(const gqa_kv8_cache_t* c, const gqa_kv8_batch_t* b, moe_status_t* st) {
  *st = MOE_ERR_INVALID_ARG;
  if (!b || !b->page_table || !b->lens || !b->offsets) return false;
  if (b->n_seqs < 1 || b->n_seqs > KV8_MAX_SEQS || b->max_pages < 1) return false;
  if (static_cast<long long>(b->max_pages) * c->page_size > (1 << 24)) return false;
  if (b->n_tokens < 0 || b->n_tokens > (1 << 20) || b->max_new < 1 || b->max_new > (1 << 20)) return false;
  *st = MOE_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(b->page_table) | reinterpret_cast<uintptr_t>(b->lens) |
       reinterpret_cast<uintptr_t>(b->offsets)) & 3u)
    return false;
  *st = MOE_OK;
  return true;
}

bool kv8_rows_ok(const void* p, long long stride, long long width, moe_status_t* st) {
  *st = MOE_ERR_INVALID_ARG;
  if (!p || stride < width || stride > (1ll << 40)) return false;
  *st = MOE_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(p) & 15u) || (stride & 7)) return false;
  *st = MOE_OK;
  return true;
}

Kv8Cache kv8_cache(const gqa_kv8_cache_t* c) {
  Kv8Cache r;
  r.codes[0] = static_cast<uint8_t*>(c->k_codes);
  r.codes[1] = static_cast<uint8_t*>(c->v_codes);
  r.scales[0] = c->k_scales;
  r.scales[1] = c->v_scales;
  r.err = c->error;
  r.n_pages = c->n_pages;
  r.page_shift = 0;
  while ((1 << r.page_shift) < c->page_size) ++r.page_shift;
  r.hkv = c->n_kv_heads;
  return r;
}

Kv8Batch kv8_batch(const gqa_kv8_batch_t* b) {
  return Kv8Batch{b->page_table, b->lens, b->offsets, b->n_seqs, b->max_pages, b->n_tokens, b->max_new};
}

namespace {

template <bool APPEND>
moe_status_t kv8_rows_launch(const gqa_kv8_cache_t* cache, const Kv8RowsParams& p, cudaStream_t s) {
  const long long warps = 2ll * p.units * p.c.hkv;
  const dim3 grid(static_cast<unsigned>((warps + KC_WARPS - 1) / KC_WARPS)), block(KC_WARPS * 32);
  void (*k)(Kv8RowsParams);
  const bool d128 = cache->head_size == 128, e4 = cache->format == GQA_KV8_E4M3;
  if (APPEND)
    k = d128 ? (e4 ? kv8_append_kernel<128, GQA_KV8_E4M3> : kv8_append_kernel<128, GQA_KV8_INT8>)
             : (e4 ? kv8_append_kernel<64, GQA_KV8_E4M3> : kv8_append_kernel<64, GQA_KV8_INT8>);
  else
    k = d128 ? (e4 ? kv8_gather_kernel<128, GQA_KV8_E4M3> : kv8_gather_kernel<128, GQA_KV8_INT8>)
             : (e4 ? kv8_gather_kernel<64, GQA_KV8_E4M3> : kv8_gather_kernel<64, GQA_KV8_INT8>);
  const cudaError_t e = launch_pdl(k, grid, block, 0, s, p);
  if (e != cudaSuccess) {
    set_error_detail(APPEND ? "gqa_kv8_append: launch" : "gqa_kv8_gather: launch", e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t gqa_kv8_append(const gqa_kv8_cache_t* cache, const gqa_kv8_batch_t* batch, const void* k,
                                       long long k_stride, const void* v, long long v_stride, moe_stream_t stream) {
  moe_status_t st;
  if (!kv8_cache_ok(cache, &st) || !kv8_batch_ok(cache, batch, &st)) return st;
  const long long width = static_cast<long long>(cache->n_kv_heads) * cache->head_size;
  if (batch->n_tokens == 0) return MOE_OK;
  if (!kv8_rows_ok(k, k_stride, width, &st) || !kv8_rows_ok(v, v_stride, width, &st)) return st;
  Kv8RowsParams p;
  std::memset(&p, 0, sizeof p);
  p.c = kv8_cache(cache);
  p.b = kv8_batch(batch);
  p.in[0] = static_cast<const __nv_bfloat16*>(k);
  p.in[1] = static_cast<const __nv_bfloat16*>(v);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.units = kv8_units(batch->n_tokens, batch->n_seqs);
  return kv8_rows_launch<true>(cache, p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t gqa_kv8_gather(const gqa_kv8_cache_t* cache, const gqa_kv8_batch_t* batch, void* k_out,
                                       void* v_out, moe_stream_t stream) {
  moe_status_t st;
  if (!kv8_cache_ok(cache, &st) || !kv8_batch_ok(cache, batch, &st)) return st;
  const long long width = static_cast<long long>(cache->n_kv_heads) * cache->head_size;
  if (batch->n_tokens == 0) return MOE_OK;
  if (!kv8_rows_ok(k_out, width, width, &st) || !kv8_rows_ok(v_out, width, width, &st)) return st;
  Kv8RowsParams p;
  std::memset(&p, 0, sizeof p);
  p.c = kv8_cache(cache);
  p.b = kv8_batch(batch);
  p.out[0] = static_cast<__nv_bfloat16*>(k_out);
  p.out[1] = static_cast<__nv_bfloat16*>(v_out);
  p.units = kv8_units(batch->n_tokens, batch->n_seqs);
  return kv8_rows_launch<false>(cache, p, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" moe_status_t gqa_kv8_get_error(const gqa_kv8_cache_t* cache) {
  if (!cache || !cache->error) return MOE_ERR_INVALID_ARG;
  unsigned v = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&v, cache->error, 4, cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && v) e = cudaMemset(cache->error, 0, 4);
  if (e == cudaSuccess && v) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    set_error_detail("gqa_kv8_get_error", e);
    return MOE_ERR_CUDA;
  }
  if (v & ERRBIT_TIMEOUT) return MOE_ERR_TIMEOUT;
  if (v & ERRBIT_BOUNDS) return MOE_ERR_DEVICE_BOUNDS;
  if (v & ERRBIT_NONFINITE) return MOE_ERR_NONFINITE;
  return MOE_OK;
}

extern "C" moe_status_t gqa_rope_plan_init(gqa_rope_plan_t* plan, int head_size, int rotary, double theta,
                                           const double* inv_freq, const int* sections, int n_axes, int cyclic) {
  if (!plan || n_axes < 1 || n_axes > GQA_ROPE_MAX_AXES) return MOE_ERR_INVALID_ARG;
  if (head_size != 64 && head_size != 128) return MOE_ERR_UNSUPPORTED;
  if (rotary < 16 || rotary > head_size || rotary % 16) return MOE_ERR_INVALID_ARG;
  const int half = rotary / 2;
  int left[GQA_ROPE_MAX_AXES] = {half, 0, 0, 0};
  if (sections) {
    long long sum = 0;
    for (int a = 0; a < n_axes; ++a) {
      if (sections[a] < 0) return MOE_ERR_INVALID_ARG;
      left[a] = sections[a];
      sum += sections[a];
    }
    if (sum != half) return MOE_ERR_INVALID_ARG;
  } else if (n_axes != 1) {
    return MOE_ERR_INVALID_ARG;
  }
  if (!inv_freq && !(theta > 0.0 && std::isfinite(theta))) return MOE_ERR_INVALID_ARG;
  std::memset(plan, 0, sizeof *plan);
  constexpr double two_pi = 6.283185307179586476925286766559;
  int axis = 0;
  for (int j = 0; j < half; ++j) {
    const double f = inv_freq ? inv_freq[j] : std::pow(theta, -2.0 * j / rotary);
    if (!std::isfinite(f)) return MOE_ERR_INVALID_ARG;
    const double turns = f / two_pi, part = turns - std::floor(turns);
    // 2^64 * part, in two steps so that part = 1 - tiny cannot overflow
    const double hi = std::floor(std::ldexp(part, 32));
    plan->turn[j] = (static_cast<uint64_t>(hi) << 32) + static_cast<uint64_t>(std::ldexp(std::ldexp(part, 32) - hi, 32));
    while (left[axis] == 0) axis = (axis + 1) % n_axes;   // some axis still has pairs left
    plan->axis[j] = static_cast<uint8_t>(axis);
    --left[axis];
    if (cyclic) axis = (axis + 1) % n_axes;
  }
  plan->head_size = head_size;
  plan->rotary = rotary;
  plan->n_axes = n_axes;
  return MOE_OK;
}

namespace {

moe_status_t rope_launch(const gqa_rope_plan_t* plan, const gqa_norm_t* norm, const void* q, long long q_stride, int n_q_heads,
                         const void* k, long long k_stride, int n_k_heads, const int32_t* pos, int T, void* q_out,
                         long long q_out_stride, void* k_out, long long k_out_stride, moe_stream_t stream) {
  if (!plan || T < 0 || T > (1 << 20) || n_q_heads < 1 || n_q_heads > 256 || n_k_heads < 0 || n_k_heads > 256)
    return MOE_ERR_INVALID_ARG;
  const int D = plan->head_size;
  if ((D != 64 && D != 128) || plan->rotary < 16 || plan->rotary > D || plan->rotary % 16 || plan->n_axes < 1 ||
      plan->n_axes > GQA_ROPE_MAX_AXES)
    return MOE_ERR_INVALID_ARG;
  RopeParams p;
  std::memset(&p, 0, sizeof p);
  p.half = plan->rotary / 2;
  for (int j = 0; j < p.half; ++j) {
    if (plan->axis[j] >= plan->n_axes) return MOE_ERR_INVALID_ARG;
    p.turn[j] = plan->turn[j];
    p.axis[j] = plan->axis[j];
  }
  if (norm) {
    if (!(norm->eps >= 0.0f && norm->eps <= 1e30f) || !(std::fabs(norm->offset) <= 1e30f)) return MOE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(norm->q_weight) | reinterpret_cast<uintptr_t>(norm->k_weight)) & (norm->weight_f32 ? 3u : 1u))
      return MOE_ERR_ALIGNMENT;
    p.weight[0] = norm->q_weight;
    p.weight[1] = norm->k_weight;
    p.weight_f32 = norm->weight_f32;
    p.eps = norm->eps;
    p.offset = norm->offset;
  }
  if (T == 0) return MOE_OK;
  if (!pos) return MOE_ERR_INVALID_ARG;
  moe_status_t st;
  const long long qw = static_cast<long long>(n_q_heads) * D, kw = static_cast<long long>(n_k_heads) * D;
  if (!kv8_rows_ok(q, q_stride, qw, &st) || !kv8_rows_ok(q_out, q_out_stride, qw, &st)) return st;
  if (n_k_heads && (!kv8_rows_ok(k, k_stride, kw, &st) || !kv8_rows_ok(k_out, k_out_stride, kw, &st))) return st;
  if (reinterpret_cast<uintptr_t>(pos) & 3u) return MOE_ERR_ALIGNMENT;
  if ((q == q_out && q_stride != q_out_stride) || (n_k_heads && k == k_out && k_stride != k_out_stride))
    return MOE_ERR_INVALID_ARG;
  p.in[0] = static_cast<const __nv_bfloat16*>(q);
  p.in[1] = static_cast<const __nv_bfloat16*>(k);
  p.out[0] = static_cast<__nv_bfloat16*>(q_out);
  p.out[1] = static_cast<__nv_bfloat16*>(k_out);
  p.in_stride[0] = q_stride;
  p.in_stride[1] = k_stride;
  p.out_stride[0] = q_out_stride;
  p.out_stride[1] = k_out_stride;
  p.heads[0] = n_q_heads;
  p.heads[1] = n_k_heads;
  p.pos = pos;
  p.T = T;
  p.n_axes = plan->n_axes;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  // One token per CTA spreads few tokens over more SMs, four share the launch of a CTA and its wait
  // for the sines (18 heads of 128): 64 tokens 2.1 us one by one and 2.7 by four, 512 2.6 and 2.8,
  // 1024 4.1 and 3.7, 2048 5.8 and 5.2, 16384 43.6 and 28.3.
  p.tokens = T >= 1024 ? 4 : 1;
  // With norms, as many as make whole waves of CTAs, as few as there can be with NR_TOKENS at most:
  // 16384 tokens 29.6 us in one wave of 27 each, 31.3 in three of 9, 33.6 in four of 7.
  constexpr int wave = 152 * NR_CTAS;
  if (norm) p.tokens = (T - 1) / (wave * ((T - 1) / (wave * NR_TOKENS) + 1)) + 1;
  const int ng = 512 / D, per = norm ? (n_q_heads + ng - 1) / ng + (n_k_heads + ng - 1) / ng : n_q_heads + n_k_heads;
  p.inv_heads = ((1u << 21) + per - 1) / per;
  const dim3 grid((T + p.tokens - 1) / p.tokens);
  const size_t smem = ((norm ? 3ull : 2ull) * p.tokens * p.half + (norm ? 2 * D : 0)) * sizeof(float);
  auto* kernel = norm ? (D == 128 ? norm_rope_kernel<128> : norm_rope_kernel<64>)
                      : (D == 128 ? rope_kernel<128> : rope_kernel<64>);
  e = launch_pdl(kernel, grid, dim3(RP_THREADS), smem, s, p);
  if (e != cudaSuccess) {
    set_error_detail(norm ? "gqa_norm_rope: launch" : "gqa_rope: launch", e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace

extern "C" moe_status_t gqa_rope(const gqa_rope_plan_t* plan, const void* q, long long q_stride, int n_q_heads,
                                 const void* k, long long k_stride, int n_k_heads, const int32_t* pos, int T,
                                 void* q_out, long long q_out_stride, void* k_out, long long k_out_stride,
                                 moe_stream_t stream) {
  return rope_launch(plan, nullptr, q, q_stride, n_q_heads, k, k_stride, n_k_heads, pos, T, q_out, q_out_stride, k_out,
                     k_out_stride, stream);
}

extern "C" moe_status_t gqa_norm_rope(const gqa_rope_plan_t* plan, const gqa_norm_t* norm, const void* q, long long q_stride,
                                      int n_q_heads, const void* k, long long k_stride, int n_k_heads, const int32_t* pos,
                                      int T, void* q_out, long long q_out_stride, void* k_out, long long k_out_stride,
                                      moe_stream_t stream) {
  if (!norm) return MOE_ERR_INVALID_ARG;
  return rope_launch(plan, norm, q, q_stride, n_q_heads, k, k_stride, n_k_heads, pos, T, q_out, q_out_stride, k_out,
                     k_out_stride, stream);
}
