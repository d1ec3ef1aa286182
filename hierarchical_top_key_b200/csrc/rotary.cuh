// rotary.cuh - rotary positions, alone and behind the norm of each head.
//
// A row x of one (token, head) has `dim` features.  With a norm, features
// [0, norm_dim) become
//     rms    y = x * rsqrt(mean(x^2) + eps) * weight
//     layer  y = (x - mean(x)) * rsqrt(var(x) + eps) * weight + bias
// (the rest pass unchanged), then the pairs of features [offset, offset + rot)
// turn by the token's position,
//     (a, b) -> amplitude * (a cos - b sin, b cos + a sin),
//     angle = position * inv_freq[i],   i = 0 .. rot/2 - 1,
// a and b being features 2i and 2i+1 (interleaved) or i and i + rot/2 (half).
// All of it in fp32, rounded once to the row's type.
//
// The angle needs more than fp32: at position 10^6 an fp32 product is off by
// 0.06 rad.  inv_freq / 2 pi is therefore held as a 64-bit fixed-point part of
// a turn, and position * that (modulo 2^64, an integer multiplication) is the
// phase exactly; its top 32 bits are the angle in [-1, 1) half turns that
// sincospi takes.
#pragma once
#include "common.cuh"

namespace hisa {

enum : int { NORM_NONE = 0, NORM_RMS = HISA_NORM_RMS, NORM_LAYER = HISA_NORM_LAYER };
constexpr int kRotaryMaxDim = 1024;

struct RotaryParams {
  const void* x;
  void* out;
  const int32_t* pos;        // [tokens]
  const double* inv_freq;    // [rot / 2], radians per position
  const float* weight;       // [norm_dim]
  const float* bias;         // [norm_dim] or NULL
  int64_t x_token, x_head, out_token, out_head;   // strides in elements
  int64_t rows;              // tokens * heads
  int heads, dim, rot, offset, norm_dim;
  int first, last;           // features [first, last) are written
  float amplitude, eps, sign;   // sign: -1 turns back
  bool interleaved;
};

// inv_freq (radians per position) as a fixed-point part of a turn.
__device__ __forceinline__ uint64_t turns64(double inv_freq) {
  const double t = inv_freq * 0.15915494309189533577;            // 1 / (2 pi)
  return static_cast<uint64_t>(__double2ull_rn((t - floor(t)) * 18446744073709551616.0));
}

// (cos, sin) of position * frequency, times the amplitude; sign -1 turns back.
__device__ __forceinline__ float2 turn_of(int32_t pos, uint64_t turns, float amplitude, float sign) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * turns;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c * amplitude, s * amplitude * sign);
}

template <int DT> __device__ __forceinline__ float load_elem(const void* p, int64_t i);
template <> __device__ __forceinline__ float load_elem<DT_F32>(const void* p, int64_t i) {
  return static_cast<const float*>(p)[i];
}
template <> __device__ __forceinline__ float load_elem<DT_BF16>(const void* p, int64_t i) {
  return bf16_bits_to_float(static_cast<const uint16_t*>(p)[i]);
}
template <int DT> __device__ __forceinline__ void store_elem(void* p, int64_t i, float v);
template <> __device__ __forceinline__ void store_elem<DT_F32>(void* p, int64_t i, float v) {
  static_cast<float*>(p)[i] = v;
}
template <> __device__ __forceinline__ void store_elem<DT_BF16>(void* p, int64_t i, float v) {
  static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kRotaryWarps = 4;

// One warp per row, any strides, sizes and alignment: the row goes through
// shared memory in fp32.
template <int DT, int NORM>
__global__ void __launch_bounds__(32 * kRotaryWarps) norm_rotary_rows_kernel(const RotaryParams p) {
  __shared__ float buf[kRotaryWarps][kRotaryMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRotaryWarps + warp;
  if (row >= p.rows) return;
  float* b = buf[warp];
  const int64_t token = row / p.heads;
  const int head = static_cast<int>(row - token * p.heads);
  const int64_t xi = token * p.x_token + head * p.x_head, oi = token * p.out_token + head * p.out_head;
  for (int j = p.first + lane; j < p.last; j += 32) b[j] = load_elem<DT>(p.x, xi + j);
  __syncwarp();
  if (NORM != NORM_NONE) {
    float mean = 0.f, sq = 0.f;
    if (NORM == NORM_LAYER) {
      for (int j = lane; j < p.norm_dim; j += 32) mean += b[j];
      mean = warp_sum(mean) / static_cast<float>(p.norm_dim);
    }
    for (int j = lane; j < p.norm_dim; j += 32) sq += (b[j] - mean) * (b[j] - mean);
    const float r = 1.f / sqrtf(warp_sum(sq) / static_cast<float>(p.norm_dim) + p.eps);
    for (int j = lane; j < p.norm_dim; j += 32) {
      float y = (b[j] - mean) * r * p.weight[j];
      if (NORM == NORM_LAYER && p.bias) y += p.bias[j];
      b[j] = y;
    }
    __syncwarp();
  }
  const int half = p.rot / 2;
  const int32_t pos = p.pos[token];
  for (int i = lane; i < half; i += 32) {
    const float2 t = turn_of(pos, turns64(p.inv_freq[i]), p.amplitude, p.sign);
    const int ja = p.offset + (p.interleaved ? 2 * i : i), jb = p.interleaved ? ja + 1 : ja + half;
    const float va = b[ja], vb = b[jb];
    b[ja] = va * t.x - vb * t.y;
    b[jb] = vb * t.x + va * t.y;
  }
  __syncwarp();
  for (int j = p.first + lane; j < p.last; j += 32) store_elem<DT>(p.out, oi + j, b[j]);
}

}  // namespace hisa
