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
//
// The pair of CTAs of sparse_attn.cuh: 128 heads are the M of every MMA, each
// CTA holds half the features (288 of the row's 576, 256 of the output's 512),
// computes its part of a 64-key tile's logits, the parts cross through
// distributed shared memory, and both run the same softmax.  What differs:
//   - the keys are not gathered by TMA but by eight warps that load a record's
//     codes, turn them into bf16 in registers (kv4.cuh) and store them in the
//     swizzled layout the MMA reads: 4-bit rows cross L2 and HBM, bf16 rows
//     exist only in shared memory;
//   - eight softmax warps instead of four, two to a head row (32 keys each);
//   - any number of heads (a slice's missing heads are zero rows), keys in
//     pages, and few queries split over the keys: part i of a row takes a
//     contiguous run of its tiles and writes an fp32 output with its own lse;
//     a second kernel joins the parts.
//
// Warp roles (18 warps):
//   warp 0       TMEM owner, logit MMA issuer (one thread)
//   warp 1       output MMA issuer (one thread)
//   warps 2..9   key producers: 8 rows of every tile each
//   warps 10..17 softmax: group g = 0, 1 (four warps each, a thread a head
//                row) has keys 32g .. 32g+31 of every tile and columns
//                128g .. 128g+127 of this CTA's output
// Every wait is bounded; a timeout sets the CTA's abort flag and the status
// word, and the peer CTA's waits on it then time out too.
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
  int slots;                 // the selection's table: a power of two >= 2 * top_k
  int slices, parts;         // slices of 128 heads; parts of a row's keys
  float scale_log2;          // |softmax scale| * log2(e)
  uint32_t q_keep, q_flip;   // the query is (q & keep) ^ flip: its sign bits for a negative scale, 0 and scale 1 for 0
  const int32_t* idx;        // [rows, top_k]
  const int32_t* page_table; // [batch, pages_per_seq]
  const uint8_t* cache;      // [num_pages, page_size, 416]
  const uint16_t* q;         // [rows, heads, 576] bf16
  uint16_t* o;               // [rows, heads, 512] bf16
  float* lse;                // [rows, heads]
  float* part_o;             // [rows, heads, parts, 512] when parts > 1
  float* part_lse;           // [rows, heads, parts]
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

// ---------------------------------------------------------------- tensor cores

constexpr int kKv4Threads = 576;
constexpr int kKv4ProdBase = 64, kKv4ProdWarps = 8;    // warps 2..9
constexpr int kKv4SoftBase = 320;                      // warps 10..17
static_assert(kKv4ProdWarps * 8 == kAttnTileN, "8 rows a producer warp");

struct Kv4Smem {
  uint64_t q_full;
  uint64_t kv_full[kAttnStages], kv_empty[kAttnStages];
  uint64_t s_full, s_empty;
  uint64_t p_full, pv_done;
  uint64_t x_full[2][2];         // partial logits of the peer CTA: [tile parity][key half]
  uint64_t pair[4];              // the two warps of a quarter of the head rows
  uint64_t drain[2];             // one per MMA issuer
  uint32_t tmem_base;
  int abort_flag;
  int scan[kKv4Threads / 32];
  float red[2][2][kAttnHeads];   // [parity][group]: a row's maximum (at the end its sum) over the group's keys
};

// The barriers and the row maxima, then the stages (1 KB aligned), the peer's
// partial logits and the record list.
constexpr size_t kKv4Head = 3 * 1024;
static_assert(sizeof(Kv4Smem) <= kKv4Head, "the head holds the barriers");
constexpr size_t kKv4SmemBytes = kKv4Head + kAttnStages * kAttnStage + 2 * kAttnHeads * kAttnTileN * 4 + kKv4MaxK * 4;
static_assert(kKv4SmemBytes <= 232448, "dynamic shared memory of one CTA");
static_assert(2 * kKv4MaxK * 4 <= kAttnStages * kAttnStage, "the selection's table fits the stages");

// A record's part of one tile row and panel: 64 codes, their four scale codes,
// and 8 positional features.
struct Kv4Piece {
  uint32_t w[8];
  uint32_t scales;
  uint4 rope;
};

__device__ __forceinline__ void kv4_load_piece(Kv4Piece& k, const uint8_t* rec, uint32_t rank, int panel) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(k.w[0]), "=r"(k.w[1]), "=r"(k.w[2]), "=r"(k.w[3]), "=r"(k.w[4]), "=r"(k.w[5]), "=r"(k.w[6]),
                 "=r"(k.w[7])
               : "l"(rec + rank * 128 + panel * 32));
  k.scales = __ldg(reinterpret_cast<const uint32_t*>(rec + kKv4ScaleAt + rank * 16 + panel * 4));
  k.rope = __ldg(reinterpret_cast<const uint4*>(rec + kKv4RopeAt + rank * 64 + panel * 16));
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__global__ void __launch_bounds__(kKv4Threads, 1) kv4_attn_kernel(const Kv4AttnParams p) {
  using namespace sm100;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Kv4Smem* sm = reinterpret_cast<Kv4Smem*>(smem_raw);
  uint8_t* kv_buf = smem_raw + kKv4Head;
  float* x_buf = reinterpret_cast<float*>(kv_buf + kAttnStages * kAttnStage);   // [2 parities][16 pieces][128 rows][4]
  int32_t* list = reinterpret_cast<int32_t*>(x_buf + 2 * kAttnHeads * kAttnTileN);
  volatile int* abort_flag = &sm->abort_flag;
  if (smem_u32(smem_raw) & 1023u) {                      // the swizzles need it; the same in every CTA
    if (threadIdx.x == 0) record_status(HISA_ERR_UNSUPPORTED);
    return;
  }

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  const int64_t item = cluster_id_x();                   // (row, head slice, part)
  const int part = static_cast<int>(item % p.parts);
  const int slice = static_cast<int>(item / p.parts % p.slices);
  const int64_t row = item / p.parts / p.slices;

  if (tid == 0) {
    mbar_init(&sm->q_full, 256);
    for (int i = 0; i < kAttnStages; ++i) {
      mbar_init(&sm->kv_full[i], kKv4ProdWarps);
      mbar_init(&sm->kv_empty[i], 1);
    }
    mbar_init(&sm->s_full, 1);
    mbar_init(&sm->s_empty, 256);
    mbar_init(&sm->p_full, 256);
    mbar_init(&sm->pv_done, 1);
    for (int i = 0; i < 2; ++i)
      for (int hf = 0; hf < 2; ++hf)
        mbar_init(&sm->x_full[i][hf], 1);   // local arrive with a half tile's bytes + the peer's st.async bytes
    for (int i = 0; i < 4; ++i) mbar_init(&sm->pair[i], 2);
    mbar_init(&sm->drain[0], 1);
    mbar_init(&sm->drain[1], 1);
    sm->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&sm->tmem_base, 512);
  const int n = kv4_select<kKv4Threads>(p, row, list, reinterpret_cast<uint32_t*>(kv_buf), p.slots, sm->scan);
  // the selection's table lies where the producers store keys for the tensor
  // cores: those stores are generic too and fenced before each hand-over
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                      // the peer's barriers exist before any remote arrive
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  // this part's run of the row's tiles
  const int T_row = (n + kAttnTileN - 1) / kAttnTileN;
  const int t0 = static_cast<int>(static_cast<int64_t>(T_row) * part / p.parts);
  const int T = static_cast<int>(static_cast<int64_t>(T_row) * (part + 1) / p.parts) - t0;
  const int first = t0 * kAttnTileN;                   // this part's first key in the list
  const int n_part = min(n - first, T * kAttnTileN);

  if (warp == 0) {
    // ------------------------------------------------------------ logit MMA issuer
    // S = q_c . k_c^T for tile k as soon as its keys are in shared memory and
    // the softmax has read tile k-1 out of the single logit buffer; the output
    // MMAs come from another thread, so these never queue behind them
    if (lane == 0) {
      constexpr uint32_t id_qk = instr_desc(kAttnHeads, kAttnTileN, 1u);
      bool ok = T == 0 || mbar_wait(&sm->q_full, 0, abort_flag);
      if (ok) tc_fence_after();
      for (int k = 0; ok && k < T; ++k) {
        const int st = k % kAttnStages;
        if (!(ok = mbar_wait(&sm->kv_full[st], static_cast<uint32_t>((k / kAttnStages) & 1), abort_flag))) break;
        if (k >= 1 && !(ok = mbar_wait(&sm->s_empty, static_cast<uint32_t>((k - 1) & 1), abort_flag))) break;
        tc_fence_after();
        const uint32_t base = smem_u32(kv_buf + st * kAttnStage);
        const uint64_t k_desc = desc_k_sw128(base);
#pragma unroll
        for (int ks = 0; ks < 4 * kAttnPanels; ++ks)
          mma_ts(tmem + kAttnTmemS, tmem + kAttnTmemQ + ks * 8,
                 k_desc + static_cast<uint64_t>((ks >> 2) * (kAttnPanelK / 16) + (ks & 3) * 2), id_qk, ks > 0 ? 1u : 0u);
        const uint64_t r_desc = desc_k_sw64(base + kAttnPanels * kAttnPanelK);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          mma_ts(tmem + kAttnTmemS, tmem + kAttnTmemQ + (4 * kAttnPanels + ks) * 8, r_desc + static_cast<uint64_t>(ks * 2),
                 id_qk, 1u);
        mma_commit(&sm->s_full);
      }
      mma_commit(&sm->drain[0]);
      mbar_drain(&sm->drain[0], 0);
    }
  } else if (warp == kAttnPvWarp) {
    // ------------------------------------------------------------ output MMA issuer
    // O_c += P . V_c for tile j once the softmax has written P_j; the tile's
    // key stage is free when this MMA completes
    if (lane == 0) {
      constexpr uint32_t id_pv = instr_desc_bmn(kAttnHeads, 256);
      bool ok = true;
      for (int j = 0; ok && j < T; ++j) {
        const int sj = j % kAttnStages;
        if (!(ok = mbar_wait(&sm->p_full, static_cast<uint32_t>(j & 1), abort_flag))) break;
        tc_fence_after();
        // V: the four 64-feature value panels of the key tile, MN-major
        const uint32_t v0 = smem_u32(kv_buf + sj * kAttnStage);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t vd = desc_mn_sw128(v0 + ks * 16 * 128, kAttnPanelK, 1024);
          mma_ts(tmem + kAttnTmemO, tmem + kAttnTmemP + ks * 8, vd, id_pv, (j > 0 || ks > 0) ? 1u : 0u);
        }
        mma_commit(&sm->kv_empty[sj]);
        mma_commit(&sm->pv_done);
      }
      mma_commit(&sm->drain[1]);
      mbar_drain(&sm->drain[1], 0);
    }
  } else if (warp < kKv4SoftBase / 32) {
    // ------------------------------------------------------------ key producers
    // Lane l has row 8w + (l & 7) and panel l >> 3 of every tile: four lanes
    // read a row's 128 consecutive code bytes, and the eight lanes of a store
    // phase hit eight rows of one panel, which the swizzle keeps in distinct
    // banks.  The next tile's record is on its way while this one is turned.
    const int r = (warp - kKv4ProdBase / 32) * 8 + (lane & 7);
    const int panel = lane >> 3;
    auto load = [&](Kv4Piece& k, int tile) {
      // past the last key: that key again, masked by the softmax
      const int e = min(tile * kAttnTileN + r, n_part - 1);
      kv4_load_piece(k, p.cache + static_cast<int64_t>(list[first + e]) * kKv4Record, rank, panel);
    };
    const uint32_t row_at = smem_u32(kv_buf) + panel * kAttnPanelK + r * 128;
    const uint32_t rope_at = smem_u32(kv_buf) + kAttnPanels * kAttnPanelK + r * 64 + ((panel ^ ((r >> 1) & 3)) << 4);
    Kv4Piece cur, nxt;
    if (T > 0) load(cur, 0);
    for (int i = 0; i < T; ++i) {
      const int st = i % kAttnStages;
      if (i + 1 < T) load(nxt, i + 1);
      int okl = 1;
      if (lane == 0)
        okl = mbar_wait(&sm->kv_empty[st], static_cast<uint32_t>(((i / kAttnStages) & 1) ^ 1), abort_flag);
      if (__shfl_sync(kFull, okl, 0) == 0) break;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint32_t s16, m24, d[4];
        kv4_scales((cur.scales >> (8 * g)) & 255u, s16, m24);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          kv4_decode8(cur.w[2 * g + u], s16, m24, d);
          sts128(row_at + st * kAttnStage + (((2 * g + u) ^ (r & 7)) << 4), d[0], d[1], d[2], d[3]);
        }
      }
      sts128(rope_at + st * kAttnStage, cur.rope.x, cur.rope.y, cur.rope.z, cur.rope.w);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->kv_full[st]);
      cur = nxt;
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3, g = (warp - kKv4SoftBase / 32) >> 2;
    const int h = quarter * 32 + lane;                 // head row = TMEM lane
    const bool head_ok = slice * kAttnHeads + h < p.heads;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    constexpr uint32_t kXBytes = kAttnHeads * kAttnTileN * 4;           // one exchange buffer
    const uint32_t peer_x = peer_addr(x_buf + (8 * g * kAttnHeads + h) * 4, peer);   // + buffer * kXBytes + piece * 2 KB
    const uint32_t peer_x_full = peer_addr(&sm->x_full[0][g], peer);    // + buffer * 16
    const float kInf = __int_as_float(0x7f800000);
    float m = -kInf, l = 0.f;
    bool ok = true;
    if (T > 0) {
      // this head's part of the query into TMEM: group g has value panels 2g
      // and 2g+1, group 0 the 32 positional features too
      const uint4* qh = reinterpret_cast<const uint4*>(p.q + ((row * p.heads) + slice * kAttnHeads + (head_ok ? h : 0)) *
                                                                 static_cast<int64_t>(kAttnDqk));
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
      for (int pn = 2 * g; pn < 2 * g + 2; ++pn) {
        uint32_t v[32];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint4 x = head_ok ? __ldg(qh + rank * 32 + pn * 8 + u) : zero;
          v[4 * u] = (x.x & p.q_keep) ^ p.q_flip;
          v[4 * u + 1] = (x.y & p.q_keep) ^ p.q_flip;
          v[4 * u + 2] = (x.z & p.q_keep) ^ p.q_flip;
          v[4 * u + 3] = (x.w & p.q_keep) ^ p.q_flip;
        }
        tmem_st32(t_lane + kAttnTmemQ + pn * 32, v);
      }
      if (g == 0) {
        uint32_t v[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 x = head_ok ? __ldg(qh + kAttnDv / 8 + rank * 4 + u) : zero;
          v[4 * u] = (x.x & p.q_keep) ^ p.q_flip;
          v[4 * u + 1] = (x.y & p.q_keep) ^ p.q_flip;
          v[4 * u + 2] = (x.z & p.q_keep) ^ p.q_flip;
          v[4 * u + 3] = (x.w & p.q_keep) ^ p.q_flip;
        }
        tmem_st16(t_lane + kAttnTmemQ + 32 * kAttnPanels, v);
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm->q_full);
    }
    // Every wait below is taken by all lanes and its outcome made
    // warp-uniform: the tcgen05 loads and stores that follow are .sync.aligned.
    //
    // The exchange of partial logits is sparse_attn.cuh's, each group with its
    // key half and barrier: a buffer is written again two tiles later, when
    // the peer's group has received all of my group's next tile, which each
    // of my threads sends after reading its row of this one.
    auto load_send = [&](float (&dst)[32], int tile) -> bool {
      if (!__all_sync(kFull, mbar_wait(&sm->s_full, static_cast<uint32_t>(tile & 1), abort_flag))) return false;
      tc_fence_after();
      uint32_t v[32];
      tmem_ld32(t_lane + kAttnTmemS + 32 * g, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; ++j) dst[j] = __uint_as_float(v[j]);
      tc_fence_before();
      mbar_arrive(&sm->s_empty);
      const int xb = tile & 1;
      if (h == 0) mbar_arrive_expect_tx(&sm->x_full[xb][g], kXBytes / 2);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        st_async_v4(peer_x + xb * kXBytes + c * (kAttnHeads * 16), dst[4 * c], dst[4 * c + 1], dst[4 * c + 2],
                    dst[4 * c + 3], peer_x_full + xb * 16);
      return true;
    };
    // The other group's value for this row; `turn` counts the exchanges.
    auto swap_pair = [&](float v, int turn, float& other) -> bool {
      sm->red[turn & 1][g][h] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->pair[quarter]);
      if (!__all_sync(kFull, mbar_wait(&sm->pair[quarter], static_cast<uint32_t>(turn & 1), abort_flag))) return false;
      other = sm->red[turn & 1][g ^ 1][h];
      return true;
    };
    float s[32], sn[32];
    if (T > 0) ok = load_send(s, 0);
    for (int i = 0; ok && i < T; ++i) {
      // 1. the peer's part of tile i, sent one tile ago
      const int xb = i & 1;
      if (!(ok = __all_sync(kFull, mbar_wait_cluster(&sm->x_full[xb][g], static_cast<uint32_t>((i >> 1) & 1),
                                                     abort_flag))))
        break;
      const float4* x4 = reinterpret_cast<const float4*>(x_buf + xb * (kAttnHeads * kAttnTileN)) + 8 * g * kAttnHeads + h;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float4 v = x4[c * kAttnHeads];
        s[4 * c + 0] += v.x; s[4 * c + 1] += v.y; s[4 * c + 2] += v.z; s[4 * c + 3] += v.w;
      }
      // 2. my part of tile i+1 out to the peer
      if (i + 1 < T && !(ok = load_send(sn, i + 1))) break;
      // 3. online softmax of tile i in the log2 domain, with the reference
      // that moves only when the maximum exceeds it by 8 (sparse_attn.cuh)
      const int nk = n_part - i * kAttnTileN - 32 * g;   // this group's keys of the tile
      if (nk < 32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) s[j] = j < nk ? s[j] : -kInf;
      }
      float mx4[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
      for (int j = 0; j < 32; ++j) mx4[j & 3] = fmaxf(mx4[j & 3], s[j]);
      float mt = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])), mo;
      if (!(ok = swap_pair(mt, i, mo))) break;
      mt = fmaxf(mt, mo) * p.scale_log2;
      const bool move = i == 0 || mt > m + 8.f;
      const float mx = move ? mt : m;
      const float corr = (i == 0) ? 0.f : (move ? fast_exp2(m - mx) : 1.f);
      float sum4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        s[j] = fast_exp2(__fmaf_rn(s[j], p.scale_log2, -mx));
        sum4[j & 3] += s[j];
      }
      l = l * corr + ((sum4[0] + sum4[1]) + (sum4[2] + sum4[3]));
      m = mx;
      // P and O belong to the previous tile's output MMA until it completes
      if (i >= 1 &&
          !(ok = __all_sync(kFull, mbar_wait(&sm->pv_done, static_cast<uint32_t>((i - 1) & 1), abort_flag))))
        break;
      tc_fence_after();
      {
        uint32_t v[16];
#pragma unroll
        for (int c = 0; c < 16; ++c) v[c] = pack_bf16x2(s[2 * c], s[2 * c + 1]);
        tmem_st16(t_lane + kAttnTmemP + 16 * g, v);
      }
      if (i >= 1 && __any_sync(kFull, corr != 1.f)) {    // rows whose maximum did not grow scale by 1
#pragma unroll 1
        for (int c0 = 128 * g; c0 < 128 * g + 128; c0 += 32) {
          uint32_t v[32];
          tmem_ld32(t_lane + kAttnTmemO + c0, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * corr);
          tmem_st32(t_lane + kAttnTmemO + c0, v);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm->p_full);
#pragma unroll
      for (int j = 0; j < 32; ++j) s[j] = sn[j];
    }
    // ---- epilogue: O / l, and lse
    const int64_t orow = row * p.heads + slice * kAttnHeads + h;
    const int col0 = static_cast<int>(rank) * 256 + 128 * g;
    float lo = 0.f;
    bool have = T > 0 && ok && swap_pair(l, T, lo);
    have = have && __all_sync(kFull, mbar_wait(&sm->pv_done, static_cast<uint32_t>((T - 1) & 1), abort_flag));
    if (have) {
      tc_fence_after();
      l += lo;
      const float inv = 1.f / l;
#pragma unroll 1
      for (int c0 = 0; c0 < 128; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(t_lane + kAttnTmemO + 128 * g + c0, v);
        tmem_wait_ld();
        if (!head_ok) continue;
        if (p.parts > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (orow * p.parts + part) * kAttnDv + col0 + c0);
#pragma unroll
          for (int q4 = 0; q4 < 8; ++q4)
            dst[q4] = make_float4(__uint_as_float(v[4 * q4]) * inv, __uint_as_float(v[4 * q4 + 1]) * inv,
                                  __uint_as_float(v[4 * q4 + 2]) * inv, __uint_as_float(v[4 * q4 + 3]) * inv);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.o + orow * kAttnDv + col0 + c0);
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(v[8 * q4 + 0]) * inv, __uint_as_float(v[8 * q4 + 1]) * inv);
            w.y = pack_bf16x2(__uint_as_float(v[8 * q4 + 2]) * inv, __uint_as_float(v[8 * q4 + 3]) * inv);
            w.z = pack_bf16x2(__uint_as_float(v[8 * q4 + 4]) * inv, __uint_as_float(v[8 * q4 + 5]) * inv);
            w.w = pack_bf16x2(__uint_as_float(v[8 * q4 + 6]) * inv, __uint_as_float(v[8 * q4 + 7]) * inv);
            dst[q4] = w;
          }
        }
      }
    } else if (T == 0 && head_ok && p.parts == 1) {
      uint4* dst = reinterpret_cast<uint4*>(p.o + orow * kAttnDv + col0);
      for (int q4 = 0; q4 < 16; ++q4) dst[q4] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (rank == 0 && g == 0 && head_ok && (have || T == 0)) {
      const float v = T == 0 ? -kInf : (m + log2f(l)) * 0.69314718055994531f;
      if (p.parts > 1) p.part_lse[orow * p.parts + part] = v;
      else p.lse[orow] = v;
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                      // no CTA leaves while its peer may still write to it
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of one (query, head): o = sum_i exp(lse_i - lse) o_i.  A part
// without keys has lse_i = -inf and no output to read.
__global__ void __launch_bounds__(128) kv4_join_kernel(const Kv4AttnParams p) {
  const int64_t orow = blockIdx.x;
  const float* pl = p.part_lse + orow * p.parts;
  float top = -__int_as_float(0x7f800000);
  for (int i = 0; i < p.parts; ++i) top = fmaxf(top, pl[i]);
  float z = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (top > -__int_as_float(0x7f800000)) {
    for (int i = 0; i < p.parts; ++i) {
      const float w = expf(pl[i] - top);
      if (w == 0.f) continue;
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + (orow * p.parts + i) * kAttnDv + threadIdx.x * 4);
      z += w;
      acc.x += w * v.x; acc.y += w * v.y; acc.z += w * v.z; acc.w += w * v.w;
    }
    const float inv = 1.f / z;
    acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
  }
  *reinterpret_cast<uint2*>(p.o + orow * kAttnDv + threadIdx.x * 4) =
      make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
  if (threadIdx.x == 0) p.lse[orow] = top + logf(z);   // -inf + log 0 = -inf for an empty set
}

}  // namespace hisa
