// kv4.cuh - the 4-bit latent cache: its record, the kernel that quantises rows
// as it writes them and the one that reads them back.
//
// One latent row (512 latent + 64 positional features, bf16, 1152 bytes) is a
// record of 416 bytes = 13 sectors of 32:
//   [0, 256)    512 codes n in -7..7, two's complement nibbles.  The 32-bit
//               word i holds features 8i .. 8i+7, the even ones in its low
//               half, the odd ones in its high half, each from the lowest
//               nibble up: feature pair k of the word is then one shift, one
//               mask-and-xor and one fma away from a packed bf16 pair.
//   [256, 288)  a scale code c for each 16 features,
//               s = (1 + (c & 7) / 8) * 2^((c >> 3) - 20)
//   [288, 416)  the 64 positional features in bf16, unchanged
// s is the smallest such value with 7 s >= max|x| of the group, so nothing is
// clipped and a value is off by at most s / 2 <= max|x| / 12.4 (9/8 is the
// largest step between scales).  n = x / s to the nearest, ties to even.  n s
// has 3 + 4 significant bits: bf16 holds it exactly, so what attention
// multiplies is what reading back returns.  A group beyond 7 * 3840 uses the
// largest scale and saturates; a NaN counts as 0.
#pragma once
#include "common.cuh"

namespace hisa {

constexpr int kKv4Latent = 512, kKv4Rope = 64, kKv4Width = kKv4Latent + kKv4Rope, kKv4Group = 16;
constexpr int kKv4ScaleAt = 256, kKv4RopeAt = 288, kKv4Record = 416;

__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// The 8 features of one code word as four packed bf16 pairs.  A nibble u of
// the two's complement n, its top bit flipped (n + 8), becomes the upper four
// mantissa bits of a bf16 in [1, 2): v = 1 + (n + 8) / 16, and n s is
// v * 16 s - 24 s.  16 s and 24 s are exact (4 and 6 significant bits), so
// is the result: the fma's one rounding changes nothing.
__device__ __forceinline__ void kv4_decode8(uint32_t w, uint32_t s16, uint32_t m24, uint32_t (&out)[4]) {
  constexpr uint32_t kMask = 0x00780078u, kFlip = 0x3FC03FC0u;
  out[0] = hfma2_bf16(((w << 3) & kMask) ^ kFlip, s16, m24);
  out[1] = hfma2_bf16(((w >> 1) & kMask) ^ kFlip, s16, m24);
  out[2] = hfma2_bf16(((w >> 5) & kMask) ^ kFlip, s16, m24);
  out[3] = hfma2_bf16(((w >> 9) & kMask) ^ kFlip, s16, m24);
}

// (16 s, -24 s) of scale code g of the four in `codes`, as packed bf16 pairs:
// the code is the exponent's low bits and the upper mantissa bits of s in
// bf16, and 16 s has its exponent 4 up.
__device__ __forceinline__ void kv4_scales(uint32_t codes, int g, uint32_t& s16, uint32_t& m24) {
  constexpr uint32_t kBias = (127u - 20u + 4u) << 7;
  s16 = __byte_perm(codes, 0u, 0x4040u + 0x0101u * g) * 16u + (kBias | (kBias << 16));
  m24 = hmul2_bf16(s16, 0xBFC0BFC0u);          // * -1.5
}

// The scale code of a group whose largest magnitude is amax (not NaN).
__device__ __forceinline__ uint32_t kv4_scale_code(float amax) {
  if (!(amax > 0.f)) return 0u;
  // the grid value at or below amax / 7, from the bits of the quotient, then
  // up while 7 s < amax: 7 s has at most 7 significant bits, so the
  // comparison is exact and the quotient's own rounding does not matter
  const int bits = __float_as_int(amax * (1.f / 7.f));
  int c = (bits >> 20) - ((127 - 20) << 3) - 1;
  c = c < 0 ? 0 : c;
  while (c < 255 && 7.f * __int_as_float((c << 20) + ((127 - 20) << 23)) < amax) ++c;
  return static_cast<uint32_t>(c > 255 ? 255 : c);
}

struct Kv4RowParams {
  const int32_t* slots;      // [n] record numbers
  uint8_t* cache;            // [num_slots, 416]
  uint8_t* rows;             // [n, 576] bf16, row_stride bytes apart
  int64_t n, num_slots, row_stride;
};

constexpr int kKv4Warps = 8;

// One warp per row, one 16-feature group per lane: the group's maximum, scale
// and codes need no other lane.  Slots below 0 are skipped (padding), slots
// past the cache are skipped and reported.
__global__ void __launch_bounds__(32 * kKv4Warps) kv4_write_kernel(const Kv4RowParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kKv4Warps + (threadIdx.x >> 5);
  if (row >= p.n) return;
  const int64_t slot = __ldg(p.slots + row);
  if (slot < 0) return;
  if (slot >= p.num_slots) {
    if (lane == 0) record_status(HISA_ERR_INVALID_ARG);
    return;
  }
  const uint8_t* src = p.rows + row * p.row_stride;
  uint8_t* dst = p.cache + slot * kKv4Record;
  const uint4 a = *reinterpret_cast<const uint4*>(src + lane * 32), b = *reinterpret_cast<const uint4*>(src + lane * 32 + 16);
  float v[16];
  Vec16<DT_BF16>::unpack(a, v);
  Vec16<DT_BF16>::unpack(b, v + 8);
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(v[j]));     // fmaxf drops a NaN
  const uint32_t code = kv4_scale_code(amax);
  const float s = __int_as_float(static_cast<int>(code << 20) + ((127 - 20) << 23));
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    // x has 8 significant bits and s four: the fp32 quotient is never rounded
    // onto a half step that x / s is not on
    float n = rintf(v[j] / s);
    n = n == n ? fminf(fmaxf(n, -7.f), 7.f) : 0.f;
    const int at = 4 * ((j & 7) >> 1) + 16 * (j & 1);
    w[j >> 3] |= (static_cast<uint32_t>(static_cast<int>(n)) & 15u) << at;
  }
  *reinterpret_cast<uint2*>(dst + lane * 8) = make_uint2(w[0], w[1]);
  dst[kKv4ScaleAt + lane] = static_cast<uint8_t>(code);
  if (lane < 8)
    *reinterpret_cast<uint4*>(dst + kKv4RopeAt + lane * 16) =
        *reinterpret_cast<const uint4*>(src + 2 * kKv4Latent + lane * 16);
}

// One warp per row, one 16-feature group per lane.  A slot below 0 gives a
// zero row, one past the cache too and is reported.
__global__ void __launch_bounds__(32 * kKv4Warps) kv4_read_kernel(const Kv4RowParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kKv4Warps + (threadIdx.x >> 5);
  if (row >= p.n) return;
  const int64_t slot = __ldg(p.slots + row);
  uint8_t* dst = p.rows + row * p.row_stride;
  uint32_t o[8] = {};
  uint4 rope = make_uint4(0u, 0u, 0u, 0u);
  if (slot >= 0 && slot < p.num_slots) {
    const uint8_t* src = p.cache + slot * kKv4Record;
    const uint2 w = *reinterpret_cast<const uint2*>(src + lane * 8);
    uint32_t s16, m24;
    kv4_scales(src[kKv4ScaleAt + lane], 0, s16, m24);
    uint32_t d[4];
    kv4_decode8(w.x, s16, m24, d);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = d[j];
    kv4_decode8(w.y, s16, m24, d);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[4 + j] = d[j];
    if (lane < 8) rope = *reinterpret_cast<const uint4*>(src + kKv4RopeAt + lane * 16);
  } else if (slot >= p.num_slots && lane == 0) {
    record_status(HISA_ERR_INVALID_ARG);
  }
  *reinterpret_cast<uint4*>(dst + lane * 32) = make_uint4(o[0], o[1], o[2], o[3]);
  *reinterpret_cast<uint4*>(dst + lane * 32 + 16) = make_uint4(o[4], o[5], o[6], o[7]);
  if (lane < 8) *reinterpret_cast<uint4*>(dst + 2 * kKv4Latent + lane * 16) = rope;
}

}  // namespace hisa
