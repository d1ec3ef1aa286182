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
// s is the smallest such value with 7 s >= max|x| of the group: nothing is
// clipped and a value is off by at most s / 2 <= max|x| / 12.4 (9/8 is the
// largest step between scales) where max|x| lies between 7 * 2^-20, below which
// the smallest scale stays and a value is off by up to 2^-21, and 7 * 3840 =
// 26880, beyond which the largest one stays and the group saturates.  n = x / s to
// the nearest, ties to even.  n s has 3 + 4 significant bits: bf16 holds it
// exactly, so what attention multiplies is what reading back returns.  A NaN
// counts as 0.
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
constexpr int kKv4Rows = 2;                    // rows of a warp, all their loads in flight together

// The 16 codes of a group with scale code `code`, two words.  n = x / s to the
// nearest even without a division: x / s, x of 8 significant bits and s of 4,
// is a half step or at least 2^-10 from one; x * (1 / s) in an fma that
// rounds to multiples of 2^-13 (the addend's unit) is therefore on the same
// side of it, and exactly there if x / s is.  Adding 1.5 * 2^23 rounds to
// even integers' bits.  Needs |x| <= 7 s.
__device__ __forceinline__ uint2 kv4_codes(const float (&v)[16], float s) {
  const float inv = 1.f / s;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float y = __fadd_rn(__fmaf_rn(v[j], inv, 1536.f), -1536.f);
    const uint32_t n = __float_as_uint(__fadd_rn(y, 12582912.f)) & 15u;
    w[j >> 3] |= n << (4 * ((j & 7) >> 1) + 16 * (j & 1));
  }
  return make_uint2(w[0], w[1]);
}

// The same with saturation, and a NaN as 0.
__device__ __forceinline__ uint2 kv4_codes_any(const float (&v)[16], float s) {
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float n = rintf(v[j] / s);
    n = n == n ? fminf(fmaxf(n, -7.f), 7.f) : 0.f;
    w[j >> 3] |= (static_cast<uint32_t>(static_cast<int>(n)) & 15u) << (4 * ((j & 7) >> 1) + 16 * (j & 1));
  }
  return make_uint2(w[0], w[1]);
}

// A warp has kKv4Rows rows, a lane one 16-feature group of each: the group's
// maximum, scale and codes need no other lane.  Bound by the 1152 + 416 bytes a
// row: 65519 rows into random slots take 23 us (4.5 TB/s; with a division an
// element and one row a warp 33).  Slots below 0 are skipped (padding), slots
// past the cache are skipped and reported.
__global__ void __launch_bounds__(32 * kKv4Warps) kv4_write_kernel(const Kv4RowParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kKv4Warps + (threadIdx.x >> 5)) * kKv4Rows;
  uint4 a[kKv4Rows], b[kKv4Rows], rope[kKv4Rows];
  int64_t slot[kKv4Rows];
#pragma unroll
  for (int u = 0; u < kKv4Rows; ++u) {
    slot[u] = row0 + u < p.n ? __ldg(p.slots + row0 + u) : -1;
    if (row0 + u >= p.n) continue;                     // a padding row is read too: the load does not wait for its slot
    const uint8_t* src = p.rows + (row0 + u) * p.row_stride;
    a[u] = __ldg(reinterpret_cast<const uint4*>(src + lane * 32));
    b[u] = __ldg(reinterpret_cast<const uint4*>(src + lane * 32 + 16));
    if (lane < 8) rope[u] = __ldg(reinterpret_cast<const uint4*>(src + 2 * kKv4Latent + lane * 16));
  }
#pragma unroll
  for (int u = 0; u < kKv4Rows; ++u) {
    if (slot[u] < 0) continue;
    if (slot[u] >= p.num_slots) {
      if (lane == 0) record_status(HISA_ERR_INVALID_ARG);
      continue;
    }
    uint8_t* dst = p.cache + slot[u] * kKv4Record;
    float v[16];
    Vec16<DT_BF16>::unpack(a[u], v);
    Vec16<DT_BF16>::unpack(b[u], v + 8);
    float amax = 0.f;
    bool odd = false;                                  // a NaN
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      amax = fmaxf(amax, fabsf(v[j]));                 // fmaxf drops a NaN
      odd |= !(v[j] == v[j]);
    }
    const uint32_t code = kv4_scale_code(amax);
    const float s = __int_as_float(static_cast<int>(code << 20) + ((127 - 20) << 23));
    const uint2 w = odd || amax > 7.f * s ? kv4_codes_any(v, s) : kv4_codes(v, s);
    *reinterpret_cast<uint2*>(dst + lane * 8) = w;
    dst[kKv4ScaleAt + lane] = static_cast<uint8_t>(code);
    if (lane < 8) *reinterpret_cast<uint4*>(dst + kKv4RopeAt + lane * 16) = rope[u];
  }
}

// A warp has kKv4Rows rows, a lane 32 bytes (16 features) of each.  A slot below
// 0 gives a zero row, one past the cache too and is reported.  131072 rows from
// random slots take 39 us (5.3 TB/s, 0.81 of the copy bandwidth; one row a warp
// 47, four 43).
__global__ void __launch_bounds__(32 * kKv4Warps) kv4_read_kernel(const Kv4RowParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * kKv4Warps + (threadIdx.x >> 5)) * kKv4Rows;
  int64_t slot[kKv4Rows];
  uint2 w[kKv4Rows];
  uint32_t code[kKv4Rows];
  uint4 rope[kKv4Rows];
#pragma unroll
  for (int u = 0; u < kKv4Rows; ++u) slot[u] = row0 + u < p.n ? __ldg(p.slots + row0 + u) : -1;
#pragma unroll
  for (int u = 0; u < kKv4Rows; ++u) {
    const bool in = slot[u] >= 0 && slot[u] < p.num_slots;
    const uint8_t* src = p.cache + (in ? slot[u] : 0) * kKv4Record;      // record 0 for a zero row: not used
    w[u] = __ldg(reinterpret_cast<const uint2*>(src + lane * 8));
    code[u] = __ldg(src + kKv4ScaleAt + lane);
    if (lane < 8) rope[u] = __ldg(reinterpret_cast<const uint4*>(src + kKv4RopeAt + lane * 16));
  }
#pragma unroll
  for (int u = 0; u < kKv4Rows; ++u) {
    if (row0 + u >= p.n) break;
    const bool in = slot[u] >= 0 && slot[u] < p.num_slots;
    if (slot[u] >= p.num_slots && lane == 0) record_status(HISA_ERR_INVALID_ARG);
    uint8_t* dst = p.rows + (row0 + u) * p.row_stride;
    uint32_t s16, m24, d[4], e[4];
    kv4_scales(code[u], 0, s16, m24);
    kv4_decode8(w[u].x, s16, m24, d);
    kv4_decode8(w[u].y, s16, m24, e);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    *reinterpret_cast<uint4*>(dst + lane * 32) = in ? make_uint4(d[0], d[1], d[2], d[3]) : zero;
    *reinterpret_cast<uint4*>(dst + lane * 32 + 16) = in ? make_uint4(e[0], e[1], e[2], e[3]) : zero;
    if (lane < 8) *reinterpret_cast<uint4*>(dst + 2 * kKv4Latent + lane * 16) = in ? rope[u] : zero;
  }
}

}  // namespace hisa
