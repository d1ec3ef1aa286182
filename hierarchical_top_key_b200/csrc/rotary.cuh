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
// a turn, and position * that (modulo 2^64, an integer multiplication) adds no
// error but the part's own: one fp64 product, up to |position| * 2^-55 turns for
// inv_freq up to 1.  The phase's top 32 bits, rounded to fp32 (up to 2^-26
// turns), are the angle in [-1, 1) half turns that sincospi takes.
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
  uint32_t head_magic, half_magic;   // n / heads, n / (rot / 2) as the upper half of n * magic, for n below 2^32 / divisor
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

// The pair (a, b) turned by t = (cos, sin).  The product with the sine is rounded
// before the sum in every kernel: a rotation in place may spread the same rows
// over the lanes in another way than one out of place, and gives the same bits.
// (A norm's sums follow the lanes: where they differ, so may its last bits.)
__device__ __forceinline__ float turn_first(float a, float b, float2 t) { return __fmaf_rn(a, t.x, -__fmul_rn(b, t.y)); }
__device__ __forceinline__ float turn_second(float a, float b, float2 t) { return __fmaf_rn(b, t.x, __fmul_rn(a, t.y)); }

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
    b[ja] = turn_first(va, vb, t);
    b[jb] = turn_second(va, vb, t);
  }
  __syncwarp();
  for (int j = p.first + lane; j < p.last; j += 32) store_elem<DT>(p.out, oi + j, b[j]);
}

// ---------------------------------------------------------------- whole vectors
//
// Rows of whole 16-byte vectors: G lanes (a power of two) hold a row in
// registers, V vectors a lane, vector k of the row in lane k mod G.  The kernel
// moves every byte once each way: 64 heads of 128, 32K tokens, bf16, out of
// place, take 167 us (6.4 TB/s, 0.98 of the measured copy bandwidth; the row
// kernel above 588).  With a norm the instructions a row cost show: 32K rows of
// 576 (bf16) 22.6 us = 3.3 TB/s, 164K fp32 rows of 128 34.9 us = 4.8 TB/s.
//   - the angles depend on the token alone: a block of some rows works out the
//     (cos, sin) of its few tokens once, in shared memory, for all their heads
//     (the first rows are on their way meanwhile);
//   - weight and bias of a lane's features stay in registers over its rows
//     where they are few (two vectors a lane), for the occupancy's sake;
//   - the partner of a half-layout pair lies rot / 2 features away.  With G as
//     many vectors as that it is the same lane's next or last vector (PAIRS_IN_LANE);
//     otherwise it is loaded again, from L1.  All loads of a row are made
//     before its first store, so in place is safe.

template <int DT> __device__ __forceinline__ uint4 pack_vec(const float (&x)[Vec16<DT>::n]);
template <> __device__ __forceinline__ uint4 pack_vec<DT_F32>(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
template <> __device__ __forceinline__ uint4 pack_vec<DT_BF16>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT>
__device__ __forceinline__ void load_features(float (&w)[Vec16<DT>::n], const float* src) {
#pragma unroll
  for (int e = 0; e + 4 <= Vec16<DT>::n; e += 4) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(src + e));
    w[e] = f.x; w[e + 1] = f.y; w[e + 2] = f.z; w[e + 3] = f.w;
  }
}

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTable = 4096;             // (cos, sin) pairs of a block

enum : int { PAIRS_INTERLEAVED, PAIRS_RELOAD, PAIRS_IN_LANE };

// Blocks an SM: enough loads in flight to keep HBM busy.  Chosen on the prompt
// sizes named above.  At these register caps some bf16 kernels spill (layer norms
// with PAIRS_RELOAD 24 to 144 bytes, RMS norms with it up to 56, layer norms with
// PAIRS_IN_LANE 48, rotations in half layout 24; fp32 up to 24); they have not
// been timed at other caps.
constexpr int rotary_blocks(int norm, int v) { return v > 5 ? 2 : v > 4 ? 3 : v > 2 ? 4 : norm == NORM_NONE ? 6 : 4; }

template <int DT, int NORM, int V, int PAIRS>
__global__ void __launch_bounds__(kRotaryThreads, rotary_blocks(NORM, V)) norm_rotary_vec_kernel(const RotaryParams p, int log_g, int nvec,
                                                                         int rows_per_block) {
  constexpr int E = Vec16<DT>::n, ES = Elem<DT>::bytes;
  constexpr bool kKeep = NORM != NORM_NONE && V <= 2;  // weights in registers
  extern __shared__ __align__(16) uint8_t rot_smem[];
  const int half = p.rot / 2;
  uint64_t* turns = reinterpret_cast<uint64_t*>(rot_smem);
  float2* cs = reinterpret_cast<float2*>(turns + half);
  const int tid = threadIdx.x, G = 1 << log_g, lane = tid & (G - 1);
  const int64_t row_lo = static_cast<int64_t>(blockIdx.x) * rows_per_block;
  const int nrows = static_cast<int>(min(static_cast<int64_t>(rows_per_block), p.rows - row_lo));
  const int64_t tok_lo = row_lo / p.heads;
  const int head_lo = static_cast<int>(row_lo - tok_lo * p.heads);
  const int ntok = (head_lo + nrows - 1) / p.heads + 1;

  // row r of the block: its vectors, and the partners that other lanes hold
  uint4 raw[V], mate[PAIRS == PAIRS_RELOAD ? V : 1];
  bool live = false;
  int tk = 0;
  uint8_t* outr = nullptr;
  auto load = [&](int r) {
    live = r < nrows;
    const int at = head_lo + (live ? r : 0);
    tk = p.heads == 1 ? at : static_cast<int>(__umulhi(static_cast<uint32_t>(at), p.head_magic));
    const int head = at - tk * p.heads;
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + ((tok_lo + tk) * p.x_token + head * p.x_head) * ES;
    outr = static_cast<uint8_t*>(p.out) + ((tok_lo + tk) * p.out_token + head * p.out_head) * ES;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int k = lane + v * G, j = p.first + k * E, jr = j - p.offset;
      if (!live || k >= nvec) continue;
      raw[v] = *reinterpret_cast<const uint4*>(xr + j * ES);
      if (PAIRS == PAIRS_RELOAD && jr >= 0 && jr < p.rot)
        mate[PAIRS == PAIRS_RELOAD ? v : 0] = *reinterpret_cast<const uint4*>(xr + (jr < half ? j + half : j - half) * ES);
    }
  };
  load(tid >> log_g);

  float w[kKeep ? V : 1][E], b[kKeep && NORM == NORM_LAYER ? V : 1][E];
  if (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int j = (lane + v * G) * E;                // a norm's rows start at feature 0
      if (j >= p.norm_dim) continue;
      load_features<DT>(w[v], p.weight + j);
      if (NORM == NORM_LAYER) {
#pragma unroll
        for (int e = 0; e < E; ++e) b[v][e] = 0.f;
        if (p.bias) load_features<DT>(b[v], p.bias + j);
      }
    }
  }
  for (int i = tid; i < half; i += kRotaryThreads) turns[i] = turns64(p.inv_freq[i]);
  __syncthreads();
  for (int e = tid; e < ntok * half; e += kRotaryThreads) {
    const int t = static_cast<int>(__umulhi(static_cast<uint32_t>(e), p.half_magic));
    cs[e] = turn_of(__ldg(p.pos + tok_lo + t), turns[e - t * half], p.amplitude, p.sign);
  }
  __syncthreads();

  const int step = kRotaryThreads >> log_g;
  for (int r0 = 0; r0 < nrows; r0 += step) {           // the same trips for a warp's every group: they shuffle together
    float mean = 0.f, rs = 1.f;
    if (NORM != NORM_NONE) {
      const float inv_n = 1.f / static_cast<float>(p.norm_dim);
      if (NORM == NORM_LAYER) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int k = lane + v * G;
          if (!live || k >= nvec || k * E >= p.norm_dim) continue;
          float x[E];
          Vec16<DT>::unpack(raw[v], x);
#pragma unroll
          for (int e = 0; e < E; ++e) mean += x[e];
        }
        for (int o = G >> 1; o; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
        mean *= inv_n;
      }
      float sq = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = lane + v * G;
        if (!live || k >= nvec || k * E >= p.norm_dim) continue;
        float x[E];
        Vec16<DT>::unpack(raw[v], x);
#pragma unroll
        for (int e = 0; e < E; ++e) sq += NORM == NORM_LAYER ? (x[e] - mean) * (x[e] - mean) : x[e] * x[e];
      }
      for (int o = G >> 1; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
      rs = rsqrtf(sq * inv_n + p.eps);                 // off by 2 ulp at most
    }
    // features j .. j + E - 1 of vector `from`, normed (vector v's own, or its partner's)
    auto normed = [&](float (&x)[E], const uint4& from, int j, int v, bool own) {
      Vec16<DT>::unpack(from, x);
      if (NORM == NORM_NONE || j >= p.norm_dim) return;
      float wl[E], bl[E];
      if (kKeep && own) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          wl[e] = w[kKeep ? v : 0][e];
          if (NORM == NORM_LAYER) bl[e] = b[kKeep && NORM == NORM_LAYER ? v : 0][e];
        }
      } else {
        load_features<DT>(wl, p.weight + j);
        if (NORM == NORM_LAYER) {
#pragma unroll
          for (int e = 0; e < E; ++e) bl[e] = 0.f;
          if (p.bias) load_features<DT>(bl, p.bias + j);
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e)
        x[e] = NORM == NORM_LAYER ? (x[e] - mean) * rs * wl[e] + bl[e] : x[e] * rs * wl[e];
    };
    __syncwarp();                                      // every load of the row before its first store
    const float2* turn = cs + tk * half;
    if (PAIRS == PAIRS_IN_LANE) {
#pragma unroll
      for (int v = 0; v < V; v += 2) {
        const int k = lane + v * G, j = p.first + k * E, jr = j - p.offset;
        if (!live || k >= nvec) continue;
        float x[E], m[E];
        const bool two = k + G < nvec;
        normed(x, raw[v], j, v, true);
        if (two) normed(m, raw[v + 1], j + G * E, v + 1, true);
        if (jr >= 0 && jr < p.rot) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float2 t = turn[jr + e];
            const float c = x[e], d = m[e];
            x[e] = turn_first(c, d, t);
            m[e] = turn_second(c, d, t);
          }
        }
        *reinterpret_cast<uint4*>(outr + j * ES) = pack_vec<DT>(x);
        if (two) *reinterpret_cast<uint4*>(outr + (j + G * E) * ES) = pack_vec<DT>(m);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int k = lane + v * G, j = p.first + k * E, jr = j - p.offset;
        if (!live || k >= nvec) continue;
        float x[E];
        normed(x, raw[v], j, v, true);
        if (jr >= 0 && jr < p.rot) {
          if (PAIRS == PAIRS_INTERLEAVED) {
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              const float2 t = turn[(jr + e) >> 1];
              const float c = x[e], d = x[e + 1];
              x[e] = turn_first(c, d, t);
              x[e + 1] = turn_second(c, d, t);
            }
          } else {
            float m[E];
            const bool low = jr < half;
            normed(m, mate[PAIRS == PAIRS_RELOAD ? v : 0], low ? j + half : j - half, v, false);
            const float2* tv = turn + (low ? jr : jr - half);
#pragma unroll
            for (int e = 0; e < E; ++e)                // turn_first or turn_second, without a branch
              x[e] = __fmaf_rn(x[e], tv[e].x, __fmul_rn(m[e], low ? -tv[e].y : tv[e].y));
          }
        }
        *reinterpret_cast<uint4*>(outr + j * ES) = pack_vec<DT>(x);
      }
    }
    load(r0 + step + (tid >> log_g));
  }
}

}  // namespace hisa
