// Format of the 8-bit paged key/value cache, shared by the kernels that write
// it (nvfp4_kv_append.cu) and read it (nvfp4_kv_attention.cu).
//
// A block is 16 tokens of one key/value head: 16 * D E4M3 codes and one
// exponent byte b; a code c stands for e4m3(c) * 2^(b - 127). The scale is a
// power of two because E4M3 carries its own exponent (the relative rounding
// error is 2^-4 wherever the scale puts a value, so a finer scale would gain
// nothing), and because a block whose scale grows when a token is appended is
// then rescaled exactly, but for codes that fall to E4M3's subnormals.
//
// Key block: D / W panels of [16 tokens][W bytes], W = min(D, 128). Within a
// panel the 16-byte chunks of token r's row are exchanged: chunk c lies at
// c ^ (r & 7) (W = 128) or c ^ ((r >> 1) & 3) (W = 64). That is the tensor
// cores' swizzled K-major operand, so a plain linear copy of a page stages
// it, and 16-byte fragment loads from shared memory meet no bank conflict.
// Value block: [D channels][16 tokens], the operand of the second product
// with its contraction axis (the tokens) contiguous.
#pragma once
#include <cstdint>

#include "nvfp4_common.cuh"
#include "nvfp4_internal.h"

namespace nvfp4 {
namespace kv {

constexpr int kBlock = 16;  // tokens that share a scale
// Range of the scales' exponents. The attention weighs a key by 2^(score +
// value exponent) against the heaviest one's in f32, so the exponents' span
// (96) plus the 24 binades in which a score still counts stays within f32's
// normal range.
constexpr int kExpMin = -48, kExpMax = 48;

// Byte of (token r, channel d) in a key block of D channels.
template <int D>
__device__ __forceinline__ int k_place(int r, int d) {
  constexpr int W = D < 128 ? D : 128;
  const int turn = W == 128 ? (r & 7) : ((r >> 1) & 3);
  return (d / W) * (kBlock * W) + r * W + (((((d % W) >> 4) ^ turn) << 4) | (d & 15));
}

// Smallest e with amax * 2^-e <= 448, within the range above.
__device__ __forceinline__ int scale_exponent(float amax) {
  // amax = 1.f * 2^x <= 448 * 2^e = 1.75 * 2^(8 + e)
  const uint32_t u = __float_as_uint(amax);
  const int x = (int)(u >> 23) - 127;
  const int e = x - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < kExpMin ? kExpMin : e > kExpMax ? kExpMax : e;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// What a row's products are multiplied by, apart from the blocks' scales, to give scores in the exponent of 2: queries are
// held times 2^up_e. Times a block's scale it stays below 2^128, so that a key of zeros scores zero and not no number; a
// factor beyond 2^79 leaves scores that differ at all further apart than any weight reaches.
__device__ __forceinline__ float score_factor(float scale, int up_e) {
  const float f = (scale * exp2i(-up_e)) * 1.4426950408889634f, most = exp2i(79);
  return fminf(fmaxf(f, -most), most);
}

// Two values -> two E4M3 codes (lo in the low byte), nearest, ties to even,
// saturating at 448; NaN gives 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Four codes times 2^shift, re-encoded.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float up) {
  const uint32_t lo = e4m3x2_to_f16x2(codes & 0xFFFFu), hi = e4m3x2_to_f16x2(codes >> 16);
  const float2 a = unpack2<__half>(lo), b = unpack2<__half>(hi);
  return e4m3x4(a.x * up, a.y * up, b.x * up, b.y * up);
}

// Limit of every wait of a call's kernels (2 s unless a test shortens it), and, for tests of that limit only, a flag that
// keeps every second CTA's first tile of keys from being seen to arrive, so that a wait runs out.
struct Waits {
  uint32_t limit_ns;
  int withhold;
  __device__ __forceinline__ uint32_t stalls() const { return withhold && blockIdx.x % 2 == 0 ? 1 : 0; }
};
inline Waits waits() {
  const int us = option(kOptWaitLimitUs);
  return Waits{us > 0 ? (uint32_t)us * 1000u : 2000000000u, option(kOptTestWithhold)};
}

// New tokens and tokens in all of sequence b, made safe against offsets that
// do not fit: first .. first + n lie within [0, tokens], length within what
// the table holds. There may be more new tokens than the length says: the
// first ones' positions are negative then.
struct Seq {
  int first, n, length;
};
__device__ __forceinline__ Seq sequence(const KvBatch& bt, int b) {
  Seq s;
  int end;
  if (bt.q_offsets) {
    s.first = bt.q_offsets[b];
    end = bt.q_offsets[b + 1];
  } else {
    s.first = b;
    end = b + 1;
  }
  s.length = bt.lengths[b];
  if (s.length > bt.max_length) s.length = (int)bt.max_length;
  if (s.length < 0) s.length = 0;
  if (s.first < 0) s.first = 0;
  if (end > (int)bt.tokens) end = (int)bt.tokens;
  s.n = end > s.first ? end - s.first : 0;
  return s;
}

}  // namespace kv
}  // namespace nvfp4
