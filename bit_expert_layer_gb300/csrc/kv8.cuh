// kv8.cuh -- what the kernels of the 8-bit key/value cache share: the batch as the device
// reads it, the map of 16-position blocks to work units, and the conversions between codes
// and numbers.
#pragma once

#include "common.cuh"
#include "gqa_kv8.h"

namespace moe {

constexpr int KV8_BLOCK = 16;       // positions that share a scale
constexpr int KV8_MAX_SEQS = 1024;
constexpr int KV8_MIN_EXP = -100;   // exponent of the smallest scale

struct Kv8Cache {
  uint8_t* codes[2];    // keys, values
  float* scales[2];
  uint32_t* err;
  int n_pages, page_shift, hkv;
};

struct Kv8Batch {
  const int* page_table;
  const int* lens;
  const int* offsets;
  int n_seqs, max_pages, n_tokens, max_new;
};

// One sequence of the batch, clamped to what the call's arrays hold; `bad` when something
// was out of range (a call then leaves out what it concerns).
struct Kv8Seq {
  int off, n, len;   // first row, new tokens, cached positions
  int first;         // position of the first new token (negative: the length is too short for it)
  bool bad;
};

__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8Batch& p, int page_shift, int b) {
  Kv8Seq s;
  const int o0 = __ldg(p.offsets + b), o1 = __ldg(p.offsets + b + 1), len = __ldg(p.lens + b);
  const int cap = p.max_pages << page_shift;
  s.off = min(max(o0, 0), p.n_tokens);
  const int end = min(max(o1, s.off), p.n_tokens);
  s.len = min(max(len, 0), cap);
  // a length past the page table moves no token: those past its end are left out
  s.first = max(len, 0) - (end - s.off);
  s.n = max(min(min(end - s.off, p.max_new), cap - s.first), 0);
  // offsets that contradict the call's rows do not say which row stands where
  if (s.off != o0 || end != o1) s.n = 0;
  s.bad = s.off != o0 || end != o1 || s.n != end - s.off || s.len != len;
  return s;
}

// The 16-position blocks that the new tokens of a batch touch, as work units: sequence b
// owns units offsets[b] / 16 + 2 b and up.  A sequence of n >= 1 new tokens touches at most
// n / 16 + 2 blocks, and offsets[b + 1] / 16 - offsets[b] / 16 >= n / 16 (whole divisions),
// so the ranges do not meet, whatever the lengths are; n_tokens / 16 + 2 n_seqs units
// cover the batch, and no unit needs a table made before the launch.
__host__ __device__ __forceinline__ int kv8_units(int n_tokens, int n_seqs) { return n_tokens / KV8_BLOCK + 2 * n_seqs; }

// The last sequence whose first unit is at or before u: a search by the whole warp, 32 ways
// a step (two dependent loads for 1024 sequences).
__device__ __forceinline__ int kv8_unit_seq(const Kv8Batch& p, int u) {
  const int lane = lane_id();
  int lo = 0, n = p.n_seqs;             // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    bool ok = false;
    if (lane * step < n) {
      const int o = min(max(__ldg(p.offsets + b), 0), p.n_tokens);
      ok = lane == 0 || o / KV8_BLOCK + 2 * b <= u;
    }
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, ok));
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

// ----------------------------------------------------------------- codes and numbers
// Two codes in the low half of w (the upper half with hi) -> two fp16, exactly.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_half2(uint32_t w, int hi) {
  uint32_t d;
  if constexpr (FMT == GQA_KV8_E4M3) {
    const uint16_t s = static_cast<uint16_t>(hi ? w >> 16 : w);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(s));
  } else {
    // fp16 1024 + m has m in its low bits: bytes with the sign bit flipped are code + 128
    const uint32_t x = __byte_perm(w, 0x64646464u, hi ? 0x4342 : 0x4140);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(0x64806480u));
  }
  return d;
}
// What the int8 conversion wants before it: every code's sign bit flipped.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_flip(uint32_t w) {
  return FMT == GQA_KV8_E4M3 ? w : w ^ 0x80808080u;
}

__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Four numbers already divided by the scale -> four code bytes, nearest, ties to even.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4(float a, float b, float c, float d) {
  if constexpr (FMT == GQA_KV8_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    const float v[4] = {a, b, c, d};
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = min(max(__float2int_rn(v[i]), -127), 127);
      r |= (static_cast<uint32_t>(q) & 0xFFu) << (8 * i);
    }
    return r;
  }
}

__device__ __forceinline__ uint32_t pack2_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// The exponent of a power-of-two scale.
__device__ __forceinline__ int scale_exp(float s) { return ((__float_as_int(s) >> 23) & 0xFF) - 127; }

// The smallest e >= -100 with amax <= top * 2^e, amax given by its bf16 bits (finite, sign
// cleared): top is 448 = 1.75 * 2^8 for e4m3 and 127 = 1.984375 * 2^6 for int8.
template <int FMT>
__device__ __forceinline__ int kv8_exp_of(uint32_t amax_bits) {
  const int ex = static_cast<int>(amax_bits >> 7) - 127, mant = static_cast<int>(amax_bits & 0x7Fu);
  const int e = FMT == GQA_KV8_E4M3 ? ex - 8 + (mant > 0x60) : ex - 6 + (mant > 0x7E);
  return max(e, KV8_MIN_EXP);
}

}  // namespace moe
