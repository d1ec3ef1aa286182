// kv4_attn.cuh - attention over each query's selected keys, read from the
// 4-bit latent cache (kv4.cuh).
//
// As in sparse_attn.cuh, with kv the row a record stands for: for a query t
// with selected set S_t (its index row with -1, out-of-range entries and
// repeats dropped),
//     logit[h, j] = scale * q[t, h, :] . kv[s_j, :]
//     o[t, h, :]  = sum_j softmax_j(logit[h, :]) * kv[s_j, :512]
//     lse[t, h]   = log sum_j exp(logit[h, j])          (natural log)
// and an empty set gives o = 0, lse = -inf.
#pragma once
#include "common.cuh"
#include "kv4.cuh"
#include "sparse_attn.cuh"

namespace hisa {

constexpr int kKv4MaxK = 4096;                 // longest index row

struct Kv4AttnParams {
  int64_t rows;              // batch * Q
  int Q, L, heads, top_k;
  int page_size, pages_per_seq, num_pages;
  float scale;
  const int32_t* idx;        // [rows, top_k]
  const int32_t* page_table; // [batch, pages_per_seq]
  const uint8_t* cache;      // [num_pages, page_size, 416]
  const uint16_t* q;         // [rows, heads, 576] bf16
  uint16_t* o;               // [rows, heads, 512] bf16
  float* lse;                // [rows, heads]
};

// The records of one query's selected positions, in `list` (kKv4MaxK places,
// also the scratch) in the order of the index row; returns their number.
// A hash table of places maps each position to the first place of the row
// that holds it (the result does not depend on the order of the atomics); a
// place is kept when it is that one.  A position whose page is outside the
// cache is dropped and reported.  Every thread of the block calls it; `table`
// holds `slots` >= 2 * top_k (a power of two) words, `scan` a word per warp
// and one more.
template <int THREADS>
__device__ __forceinline__ int kv4_select(const Kv4AttnParams& p, int64_t row, int32_t* list, uint32_t* table, int slots,
                                          int* scan) {
  constexpr int kPer = (kKv4MaxK + THREADS - 1) / THREADS;
  static_assert(kPer <= 32, "one keep bit per place of a thread's run");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int K = p.top_k;
  const int per = (K + THREADS - 1) / THREADS;
  const int lo = min(K, tid * per), hi = min(K, lo + per);
  const int32_t* irow = p.idx + row * K;
  const int32_t* pages = p.page_table + (row / p.Q) * p.pages_per_seq;
  const int shift = 33 - __ffs(slots);                  // 32 - log2(slots)
  for (int i = tid; i < slots / 4; i += THREADS) reinterpret_cast<uint4*>(table)[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
  for (int i = lo; i < hi; ++i) {
    const int x = __ldg(irow + i);
    list[i] = x < p.L ? x : -1;                         // negative: not a key
  }
  __syncthreads();
  int at[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    at[u] = -1;
    if (lo + u < hi) {
      const int v = list[lo + u];
      if (v >= 0) {
        // open addressing; at most top_k distinct positions in twice as many slots
        uint32_t hs = (static_cast<uint32_t>(v) * 0x9E3779B1u) >> shift;
        for (int probe = 0; probe < slots; ++probe) {
          const uint32_t prev = atomicCAS(&table[hs], ~0u, static_cast<uint32_t>(lo + u));
          if (prev == ~0u) break;
          if (list[prev] == v) {
            atomicMin(&table[hs], static_cast<uint32_t>(lo + u));
            break;
          }
          hs = (hs + 1) & (slots - 1);
        }
        at[u] = static_cast<int>(hs);
      }
    }
  }
  __syncthreads();
  uint32_t keep = 0;
  int rec[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    rec[u] = 0;
    if (at[u] >= 0 && table[at[u]] == static_cast<uint32_t>(lo + u)) {
      const int v = list[lo + u];
      const int pg = v / p.page_size;
      const int page = __ldg(pages + pg);
      if (page >= 0 && page < p.num_pages) {
        keep |= 1u << u;
        rec[u] = page * p.page_size + (v - pg * p.page_size);
      } else {
        record_status(HISA_ERR_INVALID_ARG);
      }
    }
  }
  const int cnt = __popc(keep);
  int incl = cnt;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    const int c = scan[w];
    if (w < warp) base += c;
    total += c;
  }
  int pos = base + incl - cnt;
#pragma unroll
  for (int u = 0; u < kPer; ++u)
    if (keep & (1u << u)) list[pos++] = rec[u];
  __syncthreads();
  return total;
}

// ---------------------------------------------------------------- CUDA cores

constexpr int kKv4SimtThreads = 256, kKv4SimtHeads = 8, kKv4SimtKeys = 16;
constexpr int kKv4SimtPitch = kKv4Width + 1;

inline size_t kv4_simt_smem(int slots) {
  return (kKv4SimtHeads + kKv4SimtKeys) * kKv4SimtPitch * 4 + kKv4MaxK * 4 + static_cast<size_t>(slots) * 4 + 1024;
}

// One block per (query, 8 heads): 16 keys at a time are decoded to fp32 in
// shared memory, each thread sums half a dot product, and holds 2 features of
// all 8 heads' outputs.
__global__ void __launch_bounds__(kKv4SimtThreads) kv4_attn_simt_kernel(const Kv4AttnParams p, int slots) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint32_t* table = reinterpret_cast<uint32_t*>(smem_raw);
  int32_t* list = reinterpret_cast<int32_t*>(table + slots);
  float* sq = reinterpret_cast<float*>(list + kKv4MaxK);
  float* sk = sq + kKv4SimtHeads * kKv4SimtPitch;
  __shared__ int scan[kKv4SimtThreads / 32];
  __shared__ float sp[kKv4SimtHeads][kKv4SimtKeys], sref[kKv4SimtHeads], scorr[kKv4SimtHeads], ssum[kKv4SimtHeads];
  const int tid = threadIdx.x;
  const int groups = (p.heads + kKv4SimtHeads - 1) / kKv4SimtHeads;
  const int64_t row = blockIdx.x / groups;
  const int h0 = static_cast<int>(blockIdx.x % groups) * kKv4SimtHeads;
  const int n = kv4_select<kKv4SimtThreads>(p, row, list, table, slots, scan);
  for (int i = tid; i < kKv4SimtHeads * kKv4Width; i += kKv4SimtThreads) {
    const int h = i / kKv4Width, f = i - h * kKv4Width;
    sq[h * kKv4SimtPitch + f] =
        h0 + h < p.heads ? bf16_bits_to_float(p.q[(row * p.heads + h0 + h) * kKv4Width + f]) * p.scale : 0.f;
  }
  if (tid < kKv4SimtHeads) {
    sref[tid] = -__int_as_float(0x7f800000);
    ssum[tid] = 0.f;
  }
  float acc[kKv4SimtHeads][2] = {};
  for (int k0 = 0; k0 < n; k0 += kKv4SimtKeys) {
    const int nk = min(kKv4SimtKeys, n - k0);
    __syncthreads();
    for (int i = tid; i < kKv4SimtKeys * 64; i += kKv4SimtThreads) {
      const int j = i >> 6, w = i & 63;
      float* dst = sk + j * kKv4SimtPitch;
      if (j < nk) {
        const uint8_t* rec = p.cache + static_cast<int64_t>(list[k0 + j]) * kKv4Record;
        uint32_t s16, m24, d[4];
        kv4_scales(rec[kKv4ScaleAt + (w >> 1)], s16, m24);
        kv4_decode8(reinterpret_cast<const uint32_t*>(rec)[w], s16, m24, d);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          dst[w * 8 + 2 * u] = __uint_as_float(d[u] << 16);
          dst[w * 8 + 2 * u + 1] = __uint_as_float(d[u] & 0xFFFF0000u);
        }
        dst[kKv4Latent + w] = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(rec + kKv4RopeAt)[w]);
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) dst[w * 8 + u] = 0.f;
        dst[kKv4Latent + w] = 0.f;
      }
    }
    __syncthreads();
    {
      const int h = tid >> 5, j = (tid >> 1) & 15, hf = tid & 1;
      float s = 0.f;
      for (int f = hf; f < kKv4Width; f += 2) s += sq[h * kKv4SimtPitch + f] * sk[j * kKv4SimtPitch + f];
      s += __shfl_xor_sync(kFull, s, 1);
      s = j < nk ? s : -__int_as_float(0x7f800000);
      float mx = s;
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      const float ref = fmaxf(sref[h], mx);              // the first key of a tile exists: finite unless the logits are not
      const float e = expf(s - ref);
      float sum = e;
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) sum += __shfl_xor_sync(kFull, sum, o);
      __syncwarp();
      if (hf == 0) sp[h][j] = e;
      if ((tid & 31) == 0) {
        scorr[h] = expf(sref[h] - ref);
        ssum[h] = ssum[h] * scorr[h] + sum;
        sref[h] = ref;
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kKv4SimtHeads; ++h) {
      acc[h][0] *= scorr[h];
      acc[h][1] *= scorr[h];
    }
    for (int j = 0; j < kKv4SimtKeys; ++j) {
      const float v0 = sk[j * kKv4SimtPitch + tid], v1 = sk[j * kKv4SimtPitch + tid + 256];
#pragma unroll
      for (int h = 0; h < kKv4SimtHeads; ++h) {
        acc[h][0] += sp[h][j] * v0;
        acc[h][1] += sp[h][j] * v1;
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kKv4SimtHeads; ++h) {
    if (h0 + h >= p.heads) break;
    const float inv = n > 0 ? 1.f / ssum[h] : 0.f;
    __nv_bfloat16* o = reinterpret_cast<__nv_bfloat16*>(p.o) + (row * p.heads + h0 + h) * kKv4Latent;
    o[tid] = __float2bfloat16_rn(n > 0 ? acc[h][0] * inv : 0.f);
    o[tid + 256] = __float2bfloat16_rn(n > 0 ? acc[h][1] * inv : 0.f);
    if (tid == h)
      p.lse[row * p.heads + h0 + h] = n > 0 ? sref[h] + logf(ssum[h]) : -__int_as_float(0x7f800000);
  }
}

}  // namespace hisa
