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
// 1. kv4_select_kernel turns each index row into the list of its records.
// 2. kv4_attn_kernel: 128 heads are the M of every MMA.  Their 512 fp32 output
//    columns fill an SM's TMEM, so a pair of CTAs (a cluster) shares a query:
//    CTA r holds output columns 256r .. 256r+255.  The 64-key tiles are dealt
//    out in turn: the owner of a tile computes its whole logits (K = 576) and
//    softmax weights P, and puts P (bf16, 16 KB) into its own shared memory
//    and its peer's; both add P . V for their half of the features.  Nothing
//    is computed twice, and what crosses between the SMs is 8 KB a tile each
//    way.  Producer warps load the records' codes, turn them into bf16 in
//    registers and store them in the swizzled layout the MMA reads: 4-bit rows
//    cross L2 and HBM, bf16 rows exist only in shared memory.  An owned tile
//    needs the whole row, the peer's tile only this CTA's value half.
// 3. Few queries are split over the keys: part i of a row takes a contiguous
//    run of its tiles and writes an fp32 output with its own lse;
//    kv4_join_kernel joins the parts.
//
// Measured (128 heads, 2048 keys of 64K, 1024 queries): 0.67 ms = 868 TFLOP/s,
// 0.52 of the measured bf16 burst rate; the bf16 kernel of sparse_attn.cuh takes
// 1.02 ms.  Other divisions of the work, as whole kernels: features split and
// fp32 partial logits exchanged (32 KB a tile each way) 1.08 ms; the logits
// computed by both CTAs, nothing exchanged, 0.97 ms (shared memory's data path
// is then busy 98 % of the time).  What bounds it now is the life of a tile's
// buffers: 227 KB hold two own tiles' value halves but one of the rest of a row
// and one of the peer's, so a tile's chain (keys 2K cycles, logit MMAs 1.3K,
// softmax 2.7K, output MMA 0.5K) overlaps the next one's only in part: 4.0K
// cycles a pair of tiles, 2.4K of them MMA; a change of query adds 12K.  Tried without gain: 4 or 8 warps
// on the own tiles' halves, row loads 64 bytes a lane pair, the shifts of the
// decoding as multiplications, the weights to the own memory first.
//
// Softmax reference.  P of a tile is exp2(logit - m) for a reference m per head
// row that need not be the maximum: fp32 sums and bf16 weights keep their
// relative precision at any size.  The maximum over the query's first 32 keys
// serves the whole query unless a later logit exceeds it by more than 2^64
// (sums then stay below 2^64 * 2^12 keys * 2^15, the largest value).  Only the
// warp that meets it moves its m; weights come with the m they were made with,
// and a mark where that has moved; from a query's first marked weights on, the
// output or the weights are scaled to one reference before each MMA.
//
// The weights are rounded to bf16, the type of the values they meet in an MMA (a
// second half with what the rounding lost would double the output MMAs and what
// the CTAs send): the output's error against 64 bits is up to 2.2e-3 of its
// size, where fp32 weights and one rounding of the output leave 1.7e-3.  The sums
// are of the unrounded weights, in fp32.  Scaled weights are rounded a second
// time; only those behind a reference that has moved by 2^64 are scaled.
//
// Warp roles (26 warps a CTA, a persistent pair over queries):
//   warp 0       TMEM owner, logit MMA issuer (one thread)
//   warp 1       output MMA issuer (one thread)
//   warps 2..13  producers, three teams of four: the value half of the
//                peer's tiles; the value half of the own tiles; the rest of
//                the own tiles
//   warps 14..21 softmax of the own tiles: group g has keys 32g .. 32g+31, a
//                thread a head row
//   warps 22..25 the next query, the output, and the scaling above
// Own tiles are numbered u, the peer's v, through all of a pair's queries.
// Every wait is bounded; a timeout sets the CTA's abort flag and the status
// word, and the peer CTA's waits on it then time out too.
#pragma once
#include "common.cuh"
#include "kv4.cuh"
#include "sparse_attn.cuh"

namespace hisa {

constexpr int kKv4MaxK = 4096;                 // longest index row

struct Kv4AttnParams {
  int Q, L, heads, top_k, list_ld;
  int page_size, page_shift, pages_per_seq, num_pages;   // page_shift: log2(page_size), or -1
  int slices, parts;         // slices of 128 heads; parts of a row's keys
  int64_t rows;              // (query, head) pairs of q
  int64_t row0;              // the first query of this launch (of the chunk its workspace holds)
  uint32_t items;            // (queries of this launch) * slices * parts
  float scale_log2;          // |softmax scale| * log2(e), 1 for a scale of 0
  int sign;                  // of the scale: the logits are multiplied by it unless it is 1
  const int32_t* idx;        // [rows, top_k]
  const int32_t* page_table; // [batch, pages_per_seq]
  const uint8_t* cache;      // [num_pages, page_size, 416]
  const uint16_t* q;         // [rows, heads, 576] bf16
  uint16_t* o;               // [rows, heads, 512] bf16
  float* lse;                // [rows, heads]
  int32_t* count;            // [queries of this launch]: records of each list
  int32_t* list;             // [queries of this launch, list_ld]
  float* part_o;             // [queries of this launch, heads, parts, 512] when parts > 1
  float* part_lse;           // [queries of this launch, heads, parts]
};

// The attention and the join are launched with programmatic serialisation: each
// starts while the kernel before it ends, does what does not depend on it, and
// waits here for its end.  The selection is an ordinary launch, behind all that
// was in the stream before: what the attention reads before it waits (the query)
// is complete because of that.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- selection

constexpr int kKv4SelThreads = 512, kKv4SelWarps = kKv4SelThreads / 32;
constexpr int kKv4Per = kKv4MaxK / kKv4SelThreads;        // places of an index row per thread

// Words of the dedup table: four slots a place keep the probe chains short
// (a chain is as long for a warp as for its unluckiest lane: at 1.5 slots a
// place the chains were most of the kernel's time).
__host__ __device__ inline uint32_t kv4_table_slots(int top_k) { return 4u * static_cast<uint32_t>(top_k) + 64u; }
inline size_t kv4_select_smem(int top_k) { return (kv4_table_slots(top_k) + (top_k + 3) / 4 * 4) * 4; }

// One block per query: the records of its selected positions, in the order of
// the index row.  Where the keys' bits fit into the table's memory, a bit a key
// tells whether any position repeats; mostly none does and every place is kept.
// Otherwise a hash table of places maps each position to the first place of the
// row that holds it (the result does not depend on the order of the atomics); a
// place is kept when it is that one: 64 rows of 2048 take 6.5 us by bits, 12 by
// the table.  A position whose page is outside the
// cache is dropped and reported.  Thread t has places t, t + 512, ...: all its
// loads are in flight together.
__global__ void __launch_bounds__(kKv4SelThreads) kv4_select_kernel(const Kv4AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(16) int count[kKv4Per * kKv4SelWarps], place[kKv4Per * kKv4SelWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_kernel_start();
  const int K = p.top_k;
  const int64_t row = p.row0 + blockIdx.x;
  uint32_t* table = reinterpret_cast<uint32_t*>(smem_raw);
  const uint32_t slots = kv4_table_slots(K);
  int32_t* pos = reinterpret_cast<int32_t*>(table + slots);
  const int32_t* irow = p.idx + row * K;
  const int32_t* pages = p.page_table + (row / p.Q) * p.pages_per_seq;
  int v[kKv4Per], rec[kKv4Per];
#pragma unroll
  for (int u = 0; u < kKv4Per; ++u) {
    const int at = u * kKv4SelThreads + tid;
    const int x = at < K ? __ldg(irow + at) : -1;
    v[u] = x < p.L ? x : -1;                            // negative: not a key
  }
  const bool bits = static_cast<uint32_t>(p.L) <= 32u * slots;
  auto clear = [&](uint32_t words, uint32_t with) {    // to whole vectors: slots is a multiple of 4
    for (uint32_t i = tid; i < (words + 3) / 4; i += kKv4SelThreads)
      reinterpret_cast<uint4*>(table)[i] = make_uint4(with, with, with, with);
  };
  if (bits) clear((static_cast<uint32_t>(p.L) + 31) / 32, 0u);
  else clear(slots, ~0u);
#pragma unroll
  for (int u = 0; u < kKv4Per; ++u) {
    const int at = u * kKv4SelThreads + tid;
    if (at < K) pos[at] = v[u];
    rec[u] = -1;
    if (v[u] >= 0) {
      const int pg = p.page_shift >= 0 ? v[u] >> p.page_shift : v[u] / p.page_size;
      const int page = __ldg(pages + pg);
      if (page >= 0 && page < p.num_pages) {
        rec[u] = page * p.page_size + (v[u] - pg * p.page_size);
      }
    }
  }
  __syncthreads();
  bool unique = false;
  if (bits) {
    uint32_t again = 0;
#pragma unroll
    for (int u = 0; u < kKv4Per; ++u)
      if (v[u] >= 0) again |= atomicOr(&table[v[u] >> 5], 1u << (v[u] & 31)) >> (v[u] & 31) & 1u;
    unique = __syncthreads_or(again) == 0;
    if (!unique) {
      clear(slots, ~0u);
      __syncthreads();
    }
  }
  // every round tries all open places of the thread at once; a place that
  // finds another position in its slot goes to the next.  It ends: there are
  // more slots than places.
  uint32_t open = 0;
  int at[kKv4Per];
#pragma unroll
  for (int u = 0; u < kKv4Per; ++u) {
    at[u] = -1;
    if (v[u] >= 0 && !unique) {
      open |= 1u << u;
      at[u] = static_cast<int>(__umulhi(static_cast<uint32_t>(v[u]) * 0x9E3779B1u, slots));
    }
  }
  while (open) {
    uint32_t prev[kKv4Per];
#pragma unroll
    for (int u = 0; u < kKv4Per; ++u)
      if (open >> u & 1u) prev[u] = atomicCAS(&table[at[u]], ~0u, static_cast<uint32_t>(u * kKv4SelThreads + tid));
#pragma unroll
    for (int u = 0; u < kKv4Per; ++u) {
      if (!(open >> u & 1u)) continue;
      if (prev[u] == ~0u) {
        open &= ~(1u << u);
      } else if (pos[prev[u]] == v[u]) {
        atomicMin(&table[at[u]], static_cast<uint32_t>(u * kKv4SelThreads + tid));
        open &= ~(1u << u);
      } else {
        at[u] = at[u] + 1 == static_cast<int>(slots) ? 0 : at[u] + 1;
      }
    }
  }
  __syncthreads();
  uint32_t keep = 0;
#pragma unroll
  for (int u = 0; u < kKv4Per; ++u) {
    bool k = unique ? v[u] >= 0 : at[u] >= 0 && table[at[u]] == static_cast<uint32_t>(u * kKv4SelThreads + tid);
    if (k && rec[u] < 0) {
      record_status(HISA_ERR_INVALID_ARG);
      k = false;
    }
    const uint32_t all = __ballot_sync(kFull, k);
    if (k) keep |= 1u << u;
    if (lane == 0) count[u * kKv4SelWarps + warp] = __popc(all);
  }
  __syncthreads();
  static_assert(kKv4Per * kKv4SelWarps == 128, "four counts a lane");
  if (warp == 0) {
    const int4 c = reinterpret_cast<const int4*>(count)[lane];
    int incl = c.x + c.y + c.z + c.w;
    const int mine = incl;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(kFull, incl, off);
      if (lane >= off) incl += o;
    }
    const int base = incl - mine;
    reinterpret_cast<int4*>(place)[lane] = make_int4(base, base + c.x, base + c.x + c.y, base + c.x + c.y + c.z);
    if (lane == 31) p.count[blockIdx.x] = incl;
  }
  __syncthreads();
  int32_t* out = p.list + static_cast<int64_t>(blockIdx.x) * p.list_ld;
#pragma unroll
  for (int u = 0; u < kKv4Per; ++u) {
    const uint32_t all = __ballot_sync(kFull, (keep >> u) & 1u);
    if ((keep >> u) & 1u) out[place[u * kKv4SelWarps + warp] + __popc(all & ((1u << lane) - 1u))] = rec[u];
  }
}

// ---------------------------------------------------------------- shared memory, TMEM

constexpr int kKv4Threads = 832;
constexpr int kKv4ProdBase = 64;               // warps 2..13
constexpr int kKv4SoftBase = 448;              // warps 14..21
constexpr int kKv4CorrBase = 704;              // warps 22..25

// TMEM columns: one logit tile, six of the query's nine 64-feature panels (2
// bf16 a column), the output
constexpr uint32_t kKv4TmemS = 0, kKv4TmemQ = 64, kKv4TmemO = 256;
constexpr int kKv4QPanels = 6;                 // in TMEM; the last two latent panels and the positional one in shared memory

constexpr uint32_t kKv4Panel = kAttnTileN * 128;          // 64 keys x 64 features
constexpr uint32_t kKv4QPanel = kAttnHeads * 128;         // 128 heads x 64 features
constexpr uint32_t kKv4V = 4 * kKv4Panel;                 // a tile's value half
constexpr uint32_t kKv4Kx = 5 * kKv4Panel;                // an owned tile's other half and positional panel
constexpr uint32_t kKv4P = kAttnHeads * kAttnTileN * 2;   // a tile's weights

struct Kv4Smem {
  uint64_t q_in[4][3];                         // [output warp][panel slot]: its 32 rows of a panel of the query
  uint64_t q_full, q_free, o_empty;            // a query is in place; its last own logits are done; its output has been read
  uint64_t kx_full, kx_empty, vo_full[2], vo_empty[2];   // own tiles (kx: the rest of a row)
  uint64_t vr_full, vr_empty;                  // the peer's tiles
  uint64_t s_full, s_empty;
  uint64_t p_own, p_peer, p_free;              // weights of an own tile, of a peer's tile; both CTAs have used mine
  uint64_t first_full[2];                      // the query's reference, by query parity
  uint64_t ctl, fix_done;                      // to the output warps: scale, or a query is done; their answer
  uint64_t fin_own, fin_peer, fin_free;        // a query's sums
  uint64_t drain[2];                           // one per MMA issuer
  uint32_t tmem_base;
  int abort_flag;
  int command;                                 // to the output warps
  __align__(16) uint32_t moved[2][8];                        // [own, peer][softmax warp]: 1 + the tile whose reference that warp moved
  float m_own[2][kAttnHeads], m_peer[2][kAttnHeads];   // references of the weights in place: [key half]
  float m_first[2][kAttnHeads];                // [query parity]
  float fin[2][2][2][kAttnHeads];              // [own, peer][key half][sum, reference]
};
enum : int { kKv4Done = 0, kKv4Scale = 1, kKv4First = 2, kKv4Peer = 4 };   // flags of `command`

constexpr size_t kKv4Head = 8 * 1024;
static_assert(sizeof(Kv4Smem) <= kKv4Head, "the head holds the barriers");
constexpr size_t kKv4SmemBytes = kKv4Head + 3 * kKv4QPanel + kKv4Kx + 3 * kKv4V + 2 * kKv4P;
static_assert(kKv4SmemBytes <= 232448, "dynamic shared memory of one CTA");

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// One lane of a converged warp, in a way the compiler can see: the branch it
// takes runs on the uniform datapath.  An MMA issued behind `lane == 0` costs
// its thread 45 cycles (80 beside other warps), behind this one 32, the rate of
// an M = 128, N = 64 bf16 MMA.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

// Whether the phase has completed.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t phase) {
  uint32_t ok;
  asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
               : "=r"(ok)
               : "r"(sm100::smem_u32(bar)), "r"(phase & 1)
               : "memory");
  return ok != 0;
}
// Arrive on a barrier of another CTA of the cluster (a cluster address).
__device__ __forceinline__ void mbar_arrive_remote(uint32_t addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}

// `bytes` (a multiple of 16) at the 16-byte aligned `src` towards L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ void stg256(void* dst, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Pairs of fp32 in a 64-bit register: one instruction for two (sm_100).
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Two bf16 times f, each rounded once.
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t x, float f) {
  return pack_bf16x2(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f);
}

// Arrive once on `bar` of CTA `rank` of the cluster (the same place in its
// shared memory) when all previously issued tcgen05 operations of this thread
// have completed.
__device__ __forceinline__ void mma_commit_to(uint64_t* bar, uint32_t rank) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          sm100::smem_u32(bar)),
      "h"(static_cast<uint16_t>(1u << rank))
      : "memory");
}

__device__ __forceinline__ void st_async_b32(uint32_t addr, float v, uint32_t remote_bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr),
               "r"(__float_as_uint(v)), "r"(remote_bar)
               : "memory");
}

__device__ __forceinline__ void st_async_v4u(uint32_t addr, const uint32_t (&v)[4], uint32_t remote_bar) {
  sm100::st_async_v4(addr, __uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3]),
                     remote_bar);
}

// Shared-memory descriptor of a K-major operand without swizzle, stored as
// [16-byte piece of a row][row][16 B]: 8 rows of one piece are a 128-byte core
// matrix, the next 8 rows 128 bytes on, the next piece (8 bf16 of K) `lbo` on.
__device__ __forceinline__ uint64_t desc_k_none(uint32_t smem_addr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>(128 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

// ---------------------------------------------------------------- work items

// A load that stays where it is written: the compiler moves plain ones down to
// their use, and the latency with them.  For what the selection wrote, which
// may still have been writing when this kernel started; ldg32_here for what no
// kernel in flight writes.
__device__ __forceinline__ uint32_t ld32_here(const void* src) {
  uint32_t v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(src));
  return v;
}
__device__ __forceinline__ uint32_t ldg32_here(const void* src) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(src));
  return v;
}

// A work item, one (query, head slice, part): its tiles are t = 0 .. tiles-1,
// those with t & 1 == rank are this CTA's own.  The part's keys are list[first
// .. first + n).
struct Kv4Item {
  int64_t row;               // within this launch
  int slice, part, tiles, first, n;
  __device__ __forceinline__ int own(uint32_t rank) const { return (tiles + 1 - static_cast<int>(rank)) >> 1; }
  __device__ __forceinline__ int keys_of(int t) const { return min(kAttnTileN, n - t * kAttnTileN); }
};

// A pair's items in turn, every role for itself; the next row's number of
// records is on its way while an item is worked on.
struct Kv4Walk {
  const Kv4AttnParams& p;
  uint32_t at, step;
  int count;
  __device__ __forceinline__ explicit Kv4Walk(const Kv4AttnParams& params)
      : p(params), at(sm100::cluster_id_x()), step(gridDim.x / 2), count(0) {}
  // To begin with, behind the selection, and by next().
  __device__ __forceinline__ void fetch() {
    count = at < p.items ? static_cast<int>(ld32_here(p.count + at / static_cast<uint32_t>(p.slices * p.parts))) : 0;
  }
  __device__ __forceinline__ bool next(Kv4Item& it) {
    if (at >= p.items) return false;
    const uint32_t parts = static_cast<uint32_t>(p.parts), slices = static_cast<uint32_t>(p.slices);
    const uint32_t rest = at / parts;
    it.part = static_cast<int>(at - rest * parts);
    it.row = rest / slices;
    it.slice = static_cast<int>(rest - static_cast<uint32_t>(it.row) * slices);
    const int t_row = (count + kAttnTileN - 1) / kAttnTileN;           // at most 64, as parts
    const int t0 = t_row * it.part / p.parts;
    it.tiles = t_row * (it.part + 1) / p.parts - t0;
    it.first = t0 * kAttnTileN;
    it.n = min(count - it.first, it.tiles * kAttnTileN);
    at += step;
    fetch();
    return true;
  }
};

// Half of a record's codes for one tile row and panel (64 codes and their four
// scale codes) as bf16 into 128 swizzled bytes of a panel row.
struct Kv4Piece {
  uint32_t w[8];
  uint32_t scales;
};

__device__ __forceinline__ void ldg256(uint32_t (&w)[8], const uint8_t* src) {
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(src));
}

__device__ __forceinline__ void kv4_load_piece(Kv4Piece& k, const uint8_t* rec, int panel) {
  ldg256(k.w, rec + panel * 32);
  k.scales = ldg32_here(rec + kKv4ScaleAt + panel * 4);
}

__device__ __forceinline__ const uint8_t* kv4_at(const Kv4AttnParams& p, uint32_t id) {
  return p.cache + static_cast<int64_t>(id) * kKv4Record;
}

// To the 128 bytes at `row_at` (row r of a panel), piece c at place c ^ (r & 7),
// in the order c ^ 2 panel: the codes' 16-feature groups, two words each, change
// places by the bits of `panel` instead of being indexed by it.
__device__ __forceinline__ void kv4_store_piece(const Kv4Piece& k, uint32_t row_at, int r, int panel) {
  const uint32_t at = row_at | (((r & 7) ^ (2 * panel)) << 4);
  const bool p0 = panel & 1, p1 = panel & 2;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = p0 ? k.w[i ^ 2] : k.w[i], b = p0 ? k.w[i ^ 6] : k.w[i ^ 4];
    w[i] = p1 ? b : a;
  }
  const uint32_t scales = __byte_perm(k.scales, 0u, 0x3210u ^ (0x1111u * panel));
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t s16, m24, d[4];
    kv4_scales(scales, g, s16, m24);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      kv4_decode8(w[2 * g + u], s16, m24, d);
      sts128(at ^ ((2 * g + u) << 4), d[0], d[1], d[2], d[3]);
    }
  }
}

// ---------------------------------------------------------------- the kernel

__global__ void __launch_bounds__(kKv4Threads, 1) kv4_attn_kernel(const Kv4AttnParams p,
                                                                   const __grid_constant__ CUtensorMap qmap) {
  using namespace sm100;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Kv4Smem* sm = reinterpret_cast<Kv4Smem*>(smem_raw);
  uint8_t* q_buf = smem_raw + kKv4Head;                  // [3 panels][128 rows][128 B], swizzled
  uint8_t* kx_buf = q_buf + 3 * kKv4QPanel;              // [4 latent panels of the other half, positional][64 rows][128 B]
  uint8_t* vo_buf = kx_buf + kKv4Kx;                     // [2 own tiles][4 panels][64 rows][128 B]
  uint8_t* vr_buf = vo_buf + 2 * kKv4V;                  // [4 panels][64 rows][128 B]
  uint8_t* p_own = vr_buf + kKv4V;                       // [8 pieces][128 rows][16 B]
  uint8_t* p_peer = p_own + kKv4P;
  volatile int* abort_flag = &sm->abort_flag;
  if (smem_u32(smem_raw) & 1023u) {                      // the swizzles need it; the same in every CTA
    if (threadIdx.x == 0) record_status(HISA_ERR_UNSUPPORTED);
    return;
  }

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  // bytes that the peer's softmax sends with a tile (weights, references, the
  // warps' marks) and with a query (sums and references)
  constexpr uint32_t kPBytes = kKv4P + 2 * kAttnHeads * 4 + 8 * 4, kFinBytes = 4 * kAttnHeads * 4;

  if (tid == 0) {
    for (int i = 0; i < 12; ++i) mbar_init(&sm->q_in[i / 3][i % 3], 1);
    mbar_init(&sm->q_full, 4);
    mbar_init(&sm->q_free, 1);
    mbar_init(&sm->o_empty, 4);
    mbar_init(&sm->kx_full, 4);
    mbar_init(&sm->kx_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->vo_full[i], 4);
      mbar_init(&sm->vo_empty[i], 1);
      // rank 1: a local arrive announcing the bytes + the peer's st.async; rank 0: the writing group's warps
      mbar_init(&sm->first_full[i], rank == 0 ? 4 : 1);
      mbar_init(&sm->drain[i], 1);
    }
    mbar_init(&sm->vr_full, 4);
    mbar_init(&sm->vr_empty, 1);
    mbar_init(&sm->s_full, 1);
    mbar_init(&sm->s_empty, 8);
    mbar_init(&sm->p_own, 8);
    mbar_init(&sm->p_peer, 1);                   // announced bytes + the peer's st.async
    mbar_init(&sm->p_free, 2);                   // the output MMAs of both CTAs
    mbar_init(&sm->ctl, 1);
    mbar_init(&sm->fix_done, 4);
    for (int i = 0; i < 16; ++i) sm->moved[i >> 3][i & 7] = 0;
    mbar_init(&sm->fin_own, 8);
    mbar_init(&sm->fin_peer, 1);                 // announced bytes
    mbar_init(&sm->fin_free, 8);                 // the output warps of both CTAs
    sm->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) tmem_alloc(&sm->tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync();                                      // the peer's barriers exist before any remote arrive
  let_next_kernel_start();
  tc_fence_after();
  const uint32_t tmem = sm->tmem_base;
  auto wait = [&](uint64_t* bar, uint32_t phase) -> bool {    // by all lanes, the outcome warp-uniform
    return __all_sync(kFull, mbar_wait(bar, phase & 1, abort_flag));
  };
  auto wait_peer = [&](uint64_t* bar, uint32_t phase) -> bool {   // completed by the other CTA
    return __all_sync(kFull, mbar_wait_cluster(bar, phase & 1, abort_flag));
  };
  Kv4Walk walk(p);
  Kv4Item it;
  if (warp < kKv4CorrBase / 32) {                      // the lists; the output warps have a query to load first
    wait_for_previous_kernel();
    walk.fetch();
  }
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ logit MMA issuer
    // S = q . k^T of own tile u, once its keys are in shared memory and the
    // softmax has read tile u-1 out of the single logit buffer
    if (elect_one()) {
      constexpr uint32_t id_qk = instr_desc(kAttnHeads, kAttnTileN, 1u);
      const uint64_t q_desc = desc_k_sw128(smem_u32(q_buf)), kx_desc = desc_k_sw128(smem_u32(kx_buf));
      uint32_t u = 0, live = 0;
      bool ok = true;
      while (ok && walk.next(it)) {
        const int own = it.own(rank);
        if (own == 0) continue;
        if (!(ok = mbar_wait(&sm->q_full, live & 1, abort_flag))) break;
        ++live;
        tc_fence_after();
        for (int k = 0; k < own; ++k, ++u) {
          const uint64_t vo_desc = desc_k_sw128(smem_u32(vo_buf + (u & 1) * kKv4V));
          if (!(ok = mbar_wait(&sm->kx_full, u & 1, abort_flag))) break;
          if (u >= 1 && !(ok = mbar_wait(&sm->s_empty, (u - 1) & 1, abort_flag))) break;
          tc_fence_after();
          // the positional panel and the other half's four first: their single
          // buffer is then free for the next tile while the value half's run
#pragma unroll
          for (int pn = 0; pn < 9; ++pn) {
            if (pn == 5) {
              mma_commit(&sm->kx_empty);
              if (!(ok = mbar_wait(&sm->vo_full[u & 1], (u >> 1) & 1, abort_flag))) break;
              tc_fence_after();
            }
            const uint32_t panel = pn == 0 ? 8u : pn < 5 ? 4 * peer + pn - 1 : 4 * rank + pn - 5;    // of the row
            const uint64_t kd = pn == 0  ? kx_desc + static_cast<uint64_t>(4 * (kKv4Panel / 16))
                                : pn < 5 ? kx_desc + static_cast<uint64_t>((pn - 1) * (kKv4Panel / 16))
                                         : vo_desc + static_cast<uint64_t>((pn - 5) * (kKv4Panel / 16));
            if (panel < kKv4QPanels) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma_ts(tmem + kKv4TmemS, tmem + kKv4TmemQ + panel * 32 + ks * 8, kd + static_cast<uint64_t>(ks * 2),
                       id_qk, (pn > 0 || ks > 0) ? 1u : 0u);
            } else {
              const uint64_t qd = q_desc + static_cast<uint64_t>((panel - kKv4QPanels) * (kKv4QPanel / 16));
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                mma<DT_BF16>(tmem + kKv4TmemS, qd + static_cast<uint64_t>(ks * 2), kd + static_cast<uint64_t>(ks * 2),
                             id_qk, (pn > 0 || ks > 0) ? 1u : 0u);
            }
          }
          if (!ok) break;
          mma_commit(&sm->s_full);
        }
        if (ok) mma_commit(&sm->q_free);
      }
      mma_commit(&sm->drain[0]);
      mbar_drain(&sm->drain[0], 0);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ output MMA issuer
    // O_r += P . V_r, every tile in turn; where a softmax warp has moved a
    // reference the output warps first bring output and weights to one
    if (elect_one()) {
      constexpr uint32_t id_pv = instr_desc_bmn(kAttnHeads, 256);
      uint32_t u = 0, v = 0, live = 0, fixes = 0, drains = 0;
      bool ok = true;
      mbar_arrive_expect_tx(&sm->p_peer, kPBytes);     // the first of the peer's weights
      while (ok && walk.next(it)) {
        const int tiles = it.tiles;
        if (tiles == 0) continue;
        // the previous query's output has been read
        if (live > 0 && !(ok = mbar_wait(&sm->o_empty, (live - 1) & 1, abort_flag))) break;
        ++live;
        bool scaled = false;                           // from a query's first marked tile on all are looked at
        for (int t = 0; t < tiles; ++t) {
          const bool mine = (t & 1u) == rank;
          if (!(ok = mine ? mbar_wait(&sm->p_own, u & 1, abort_flag)
                          : mbar_wait_cluster(&sm->p_peer, v & 1, abort_flag) && mbar_wait(&sm->vr_full, v & 1, abort_flag)))
            break;
          const uint4 m0 = lds128(smem_u32(sm->moved[mine ? 0 : 1])), m1 = lds128(smem_u32(sm->moved[mine ? 0 : 1] + 4));
          const uint32_t tag = (mine ? u : v) + 1;
          if (scaled || m0.x == tag || m0.y == tag || m0.z == tag || m0.w == tag || m1.x == tag || m1.y == tag || m1.z == tag ||
              m1.w == tag) {
            scaled = true;
            mma_commit(&sm->drain[1]);                 // every MMA before
            if (!(ok = mbar_wait(&sm->drain[1], drains++ & 1, abort_flag))) break;
            sm->command = kKv4Scale + (t == 0 ? kKv4First : 0) + (mine ? 0 : kKv4Peer);
            mbar_arrive(&sm->ctl);
            if (!(ok = mbar_wait(&sm->fix_done, fixes++ & 1, abort_flag))) break;
          }
          if (!mine) {
            mbar_arrive_expect_tx(&sm->p_peer, kPBytes);
            fence_proxy_async_smem();                  // the peer's generic-proxy writes before the MMA's reads
          }
          tc_fence_after();
          // V: the four 64-feature value panels of the key tile, MN-major
          const uint64_t v_desc =
              desc_mn_sw128(smem_u32(mine ? vo_buf + (u & 1) * kKv4V : vr_buf), kKv4Panel, 1024);
          const uint64_t p_desc = desc_k_none(smem_u32(mine ? p_own : p_peer), kAttnHeads * 16);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma<DT_BF16>(tmem + kKv4TmemO, p_desc + static_cast<uint64_t>(ks * (2 * kAttnHeads * 16 / 16)),
                         v_desc + static_cast<uint64_t>(ks * (16 * 128 / 16)), id_pv, (t > 0 || ks > 0) ? 1u : 0u);
          mma_commit(mine ? &sm->vo_empty[u & 1] : &sm->vr_empty);
          if (mine) {
            mma_commit(&sm->p_free);
            ++u;
          } else {
            mma_commit_to(&sm->p_free, peer);
            ++v;
          }
        }
        if (!ok) break;
        mma_commit(&sm->drain[1]);
        if (!(ok = mbar_wait(&sm->drain[1], drains++ & 1, abort_flag))) break;
        sm->command = kKv4Done;
        mbar_arrive(&sm->ctl);
      }
      mma_commit(&sm->drain[1]);
      mbar_drain(&sm->drain[1], drains & 1);
    }
  } else if (warp < kKv4SoftBase / 32) {
    // ------------------------------------------------------------ key producers
    // Lane l has panel l & 3 and a row with r & 7 = l >> 2: four lanes read a
    // row's 128 consecutive code bytes (lanes of a row further apart would
    // take a pass of the load pipe each).  The eight lanes of a store phase
    // are two rows of four panels, whose places differ only in r & 1 for the
    // same piece; so a lane takes its pieces in the order c ^ 2 panel.
    // Registers are loaded again, for the next tile, as soon as they are
    // stored, with record numbers looked up one tile before that.
    // One code for the three teams (three copies of it, and instruction
    // fetches hold up every warp).
    const int pw = warp - kKv4ProdBase / 32, team = pw >> 2;     // 0: peer's values; 1: own values; 2: own rest
    const int panel = lane & 3;
    const int r = (pw & 3) * 16 + (lane >> 2);         // and r + 8
    const uint32_t kind = team == 0 ? peer : rank;     // parity of the team's tiles
    const uint32_t code_panel = 4 * (team == 2 ? peer : rank) + panel;     // of a record
    const uint32_t out_at = smem_u32(team == 0 ? vr_buf : team == 1 ? vo_buf : kx_buf) + panel * kKv4Panel + r * 128;
    const uint32_t rope_at = smem_u32(kx_buf) + 4 * kKv4Panel + ((r * 128) | (((2 * panel) ^ (r & 7)) << 4));
    uint32_t n = 0;                                    // tiles made, through all queries
    bool ok = true;
    while (ok && walk.next(it)) {
      const int mine = it.own(kind);
      if (mine == 0) continue;
      const int32_t* list = p.list + it.row * p.list_ld + it.first;
      // the record of the tile's row rr; past the last key that key's again, masked by the softmax
      int row0 = static_cast<int>(kind) * kAttnTileN + r;
      auto record = [&](int rr) -> uint32_t { return ld32_here(list + min(row0 + rr, it.n - 1)); };
      Kv4Piece a, b;
      uint32_t ra[8], rb[8];                           // team 2: 16 of each row's 64 positional features
      uint32_t ida = record(0), idb = record(8);
#pragma unroll 1
      for (int i = -1; i < mine; ++i) {
        if (i >= 0) {
          uint32_t at = out_at;
          uint64_t* full;
          if (team == 0) {
            if (n >= 1 && !(ok = wait(&sm->vr_empty, n - 1))) break;
            full = &sm->vr_full;
          } else if (team == 1) {
            if (n >= 2 && !(ok = wait(&sm->vo_empty[n & 1], (n >> 1) - 1))) break;
            at += (n & 1) * kKv4V;
            full = &sm->vo_full[n & 1];
          } else {
            if (n >= 1 && !(ok = wait(&sm->kx_empty, n - 1))) break;
            full = &sm->kx_full;
            sts128(rope_at, ra[0], ra[1], ra[2], ra[3]);
            sts128(rope_at ^ 16u, ra[4], ra[5], ra[6], ra[7]);
            sts128(rope_at + 8 * 128, rb[0], rb[1], rb[2], rb[3]);
            sts128((rope_at + 8 * 128) ^ 16u, rb[4], rb[5], rb[6], rb[7]);
          }
          kv4_store_piece(a, at, r, panel);
          kv4_store_piece(b, at + 8 * 128, r, panel);
          fence_proxy_async_smem();
          warp_arrive(full);
          ++n;
        }
        // the addresses not before here: they wait for the record numbers
        asm volatile("" : "+r"(ida), "+r"(idb));
        const uint8_t *pa = kv4_at(p, ida), *pb = kv4_at(p, idb);
        kv4_load_piece(a, pa, code_panel);
        kv4_load_piece(b, pb, code_panel);
        if (team == 2) {
          ldg256(ra, pa + kKv4RopeAt + panel * 32);
          ldg256(rb, pb + kKv4RopeAt + panel * 32);
        }
        row0 += 2 * kAttnTileN;
        ida = record(0);
        idb = record(8);
      }
    }
  } else if (warp < kKv4CorrBase / 32) {
    // ------------------------------------------------------------ softmax of the own tiles
    const int quarter = warp & 3, g = (warp - kKv4SoftBase / 32) >> 2;
    const int h = quarter * 32 + lane;                 // head row = TMEM lane
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t p_off = 4 * g * (kAttnHeads * 16) + h * 16;      // + piece (8 keys) * 2 KB
    const uint32_t p_at = smem_u32(p_own) + p_off;
    const uint32_t peer_p = peer_addr(p_peer + p_off, peer), peer_p_bar = peer_addr(&sm->p_peer, peer);
    const uint32_t peer_m = peer_addr(&sm->m_peer[g][h], peer);
    const uint32_t peer_mark = peer_addr(&sm->moved[1][warp - kKv4SoftBase / 32], peer);
    const float kInf = __int_as_float(0x7f800000);
    uint32_t u = 0, live = 0;
    uint32_t first_phase[2] = {0, 0};
    bool ok = true;
    while (ok && walk.next(it)) {
      if (it.tiles == 0) continue;
      const int own = it.own(rank);
      const uint32_t par = live & 1;
      if (rank == 1 && own > 0 && g == 0 && h == 0) mbar_arrive_expect_tx(&sm->first_full[par], kAttnHeads * 4);
      float m = -kInf, m_first = 0.f, l = 0.f;
      for (int k = 0; k < own; ++k, ++u) {
        if (!(ok = wait(&sm->s_full, u))) break;
        tc_fence_after();
        float s[32];
        {
          uint32_t x[32];
          tmem_ld32(t_lane + kKv4TmemS + 32 * g, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(x[i]);
        }
        tc_fence_before();
        warp_arrive(&sm->s_empty);
        if (p.sign != 1) {                             // a product: at a scale of 0 a NaN or infinity becomes NaN
          const float sign = static_cast<float>(p.sign);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] *= sign;
        }
        const int nk = it.keys_of(2 * k + static_cast<int>(rank)) - 32 * g;
        if (nk < 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = i < nk ? s[i] : -kInf;
        }
        float mx4[4] = {-kInf, -kInf, -kInf, -kInf};
#pragma unroll
        for (int i = 0; i < 32; ++i) mx4[i & 3] = fmaxf(mx4[i & 3], s[i]);
        float mt = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * p.scale_log2;
        // the reference: the maximum of the query's first 32 keys, handed to
        // the other group and both of the peer's; it stays unless exceeded by 2^64
        if (k == 0) {
          if (rank == 0 && g == 0) {
            mt = fmaxf(mt, -3e38f);                    // 32 logits of -inf: weights of 0, not of exp2(-inf + inf)
            m_first = mt;
            if (it.tiles > 1)
              st_async_b32(peer_addr(&sm->m_first[par][h], peer), mt, peer_addr(&sm->first_full[par], peer));
            sm->m_first[par][h] = mt;
            warp_arrive(&sm->first_full[par]);
          } else {
            const uint32_t phase = par ? first_phase[1] : first_phase[0];
            if (!(ok = rank == 0 ? wait(&sm->first_full[par], phase) : wait_peer(&sm->first_full[par], phase))) break;
            if (par) ++first_phase[1];
            else ++first_phase[0];
            m_first = sm->m_first[par][h];
          }
          m = m_first;
        }
        if (mt > m + 64.f) {
          l *= fast_exp2(m - mt);
          m = mt;
        }
        uint32_t w[16];
        uint64_t sum2[2] = {0, 0};                     // pairs of fp32
        const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2), m2 = pack_f32x2(-m, -m);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float a, b;
          unpack_f32x2(fma_f32x2(pack_f32x2(s[2 * i], s[2 * i + 1]), scale2, m2), a, b);
          a = fast_exp2(a);
          b = fast_exp2(b);
          sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(a, b));
          w[i] = pack_bf16x2(a, b);
        }
        float sa, sb;
        unpack_f32x2(add_f32x2(sum2[0], sum2[1]), sa, sb);
        l += sa + sb;
        // both CTAs' output MMAs have read the weights before
        if (u >= 1 && !(ok = wait_peer(&sm->p_free, u - 1))) break;
        const uint32_t mark = __any_sync(kFull, m != m_first) ? u + 1 : 0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {                  // 8 keys a piece
          const uint32_t y[4] = {w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]};
          st_async_v4u(peer_p + c * (kAttnHeads * 16), y, peer_p_bar);
        }
        st_async_b32(peer_m, m, peer_p_bar);
        if (lane == 0) {
          st_async_b32(peer_mark, __uint_as_float(mark), peer_p_bar);
          sm->moved[0][warp - kKv4SoftBase / 32] = mark;
        }
        sm->m_own[g][h] = m;
#pragma unroll
        for (int c = 0; c < 4; ++c) sts128(p_at + c * (kAttnHeads * 16), w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        fence_proxy_async_smem();
        warp_arrive(&sm->p_own);
      }
      if (!ok) break;
      // this group's sums of the query, to both CTAs' output warps
      if (live > 0 && !(ok = wait_peer(&sm->fin_free, live - 1))) break;
      const uint32_t fin_bar = peer_addr(&sm->fin_peer, peer);
      st_async_b32(peer_addr(&sm->fin[1][g][0][h], peer), l, fin_bar);
      st_async_b32(peer_addr(&sm->fin[1][g][1][h], peer), m, fin_bar);
      sm->fin[0][g][0][h] = l;
      sm->fin[0][g][1][h] = m;
      warp_arrive(&sm->fin_own);
      ++live;
    }
  } else {
    // ------------------------------------------------------------ output, scaling
    const int quarter = warp & 3;
    const int h = quarter * 32 + lane;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const float kInf = __int_as_float(0x7f800000);
    const uint32_t peer_fin_free = peer_addr(&sm->fin_free, peer);
    if (h == 0) mbar_arrive_expect_tx(&sm->fin_peer, kFinBytes);      // the first of the peer's sums
    uint32_t live = 0, commands = 0, loaded = 0;       // queries put out, commands, queries handed over
    uint32_t fills = 0;                                // query loads
    bool ok = true;

    // The next query this CTA has tiles of its own for: one walk ahead.  Its
    // rows move towards L2 when it becomes the next.
    Kv4Walk ahead(p);
    Kv4Item next;
    bool waiting = false;
    int q_row = 0;                                     // of the warp's 32 rows; past the end, zeros, for heads past the last
    auto set_query = [&](int64_t item_row, int slice, bool prefetch) {
      const int h0 = slice * kAttnHeads + quarter * 32;
      const int64_t row = (p.row0 + item_row) * p.heads + h0;
      q_row = static_cast<int>(h0 < p.heads ? row : p.rows);
      if (prefetch && lane == 0 && h0 < p.heads)
        prefetch_l2_bulk(p.q + row * kAttnDqk, min(32, p.heads - h0) * kAttnDqk * 2);
    };
    auto find_query = [&]() {
      while ((waiting = ahead.next(next)) && next.own(rank) == 0) {}
      if (waiting) set_query(next.row, next.slice, true);
    };
    // Panel pn of the warp's 32 rows into shared memory; no other warp reads or
    // writes them.  (Rows past the last head may be the next query's: their
    // results go nowhere.)
    auto query_panel = [&](int pn) {
      if (lane != 0) return;
      uint64_t* bar = &sm->q_in[quarter][pn % 3];
      mbar_arrive_expect_tx(bar, 32 * 128);
      tma_load_2d(q_buf + pn % 3 * kKv4QPanel + quarter * 32 * 128, &qmap, bar, pn * 64, q_row);
    };
    auto panel_here = [&](int pn) {                    // after an abort too: the copy is not left in flight
      uint64_t* bar = &sm->q_in[quarter][pn % 3];
      const uint32_t parity = (3 * fills + pn / 3) & 1;
      if (!mbar_wait(bar, parity, abort_flag)) mbar_drain(bar, parity);
      __syncwarp();
    };
    // The query's rows, behind the last own logits of the one before: the first
    // six panels go on into TMEM, three in flight, the last three stay.
    auto load_query = [&]() {
      tc_fence_after();
      for (int pn = 0; pn < 3; ++pn) query_panel(pn);
#pragma unroll 1
      for (int pn = 0; pn < kKv4QPanels; ++pn) {
        panel_here(pn);
        const uint32_t row_at = smem_u32(q_buf) + pn % 3 * kKv4QPanel + h * 128;
        uint32_t x[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 y = lds128(row_at + ((i ^ (h & 7)) << 4));
          x[4 * i] = y.x; x[4 * i + 1] = y.y; x[4 * i + 2] = y.z; x[4 * i + 3] = y.w;
        }
        tmem_st32(t_lane + kKv4TmemQ + pn * 32, x);
        __syncwarp();
        query_panel(pn + 3);
      }
#pragma unroll 1
      for (int pn = kKv4QPanels; pn < 9; ++pn) panel_here(pn);
      tmem_wait_st();
      fence_proxy_async_smem();
      tc_fence_before();
      ++fills;
    };
    auto hand_over = [&]() {
      warp_arrive(&sm->q_full);
      ++loaded;
      find_query();
    };
    // The first item's query does not depend on the selection: it is loaded
    // while that runs, and used unless the item turns out to have no tile here.
    // (Whatever wrote it is done: the selection, an ordinary launch, began after.)
    const uint32_t first_item = walk.at, first_rest = first_item / static_cast<uint32_t>(p.parts);
    set_query(first_rest / static_cast<uint32_t>(p.slices), static_cast<int>(first_rest % static_cast<uint32_t>(p.slices)), false);
    load_query();
    wait_for_previous_kernel();
    walk.fetch();
    ahead.fetch();
    find_query();
    if (waiting && ahead.at == first_item + ahead.step) hand_over();
    auto timed_out = [&](uint64_t t0) -> bool {        // or the CTA is aborting, warp-uniform
      bool out = *abort_flag != 0;
      if (!out && globaltimer() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        record_status(HISA_ERR_TIMEOUT);
        out = true;
      }
      return __any_sync(kFull, out);
    };

    while (ok && walk.next(it)) {
      const bool head_ok = it.slice * kAttnHeads + h < p.heads;
      const int64_t orow = it.row * p.heads + it.slice * kAttnHeads + h;      // within this launch
      uint16_t* out = p.o + (p.row0 * p.heads + orow) * kAttnDv + rank * 256;
      if (it.tiles == 0) {
        if (head_ok && p.parts == 1) {
          const uint32_t zero[8] = {};
          for (int i = 0; i < 16; ++i) stg256(out + 16 * i, zero);
        }
        if (rank == 0 && head_ok) {
          if (p.parts > 1) p.part_lse[orow * p.parts + it.part] = -kInf;
          else p.lse[p.row0 * p.heads + orow] = -kInf;
        }
        continue;
      }
      bool scaled = false;
      float mo = 0.f;                                  // what the output rows are relative to, once `scaled`
      uint64_t t0 = globaltimer();
      while (true) {
        // the next query as soon as its place is free: the output's rest is
        // then made while its first logits are.  A command may come first, and
        // may be what that place waits for.
        if (waiting) {
          bool command_here, free_here;
          for (int k = 0;; ++k) {
            command_here = __all_sync(kFull, mbar_test(&sm->ctl, commands));
            free_here = __all_sync(kFull, loaded == 0 || mbar_test(&sm->q_free, loaded - 1));
            if (command_here || free_here || ((k & 63) == 63 && !(ok = !timed_out(t0)))) break;
            __nanosleep(400);
          }
          if (!ok) break;
          if (!command_here) {
            load_query();
            hand_over();
            t0 = globaltimer();
            continue;
          }
        } else if (!(ok = wait(&sm->ctl, commands))) {
          break;
        }
        t0 = globaltimer();
        ++commands;
        const int command = *reinterpret_cast<volatile int*>(&sm->command);
        if (command == kKv4Done) break;
        const bool from_peer = (command & kKv4Peer) != 0;
        const float ma = from_peer ? sm->m_peer[0][h] : sm->m_own[0][h], mb = from_peer ? sm->m_peer[1][h] : sm->m_own[1][h];
        const float m = fmaxf(ma, mb);
        if (command & kKv4First) mo = m;
        else if (!scaled) mo = sm->m_first[live & 1][h];
        scaled = true;
        if (!(command & kKv4First) && __any_sync(kFull, m > mo)) {     // the output moves up to this tile's reference
          tc_fence_after();
          const float f = m > mo ? fast_exp2(mo - m) : 1.f;
#pragma unroll 1
          for (int c0 = 0; c0 < 256; c0 += 32) {
            uint32_t x[32];
            tmem_ld32(t_lane + kKv4TmemO + c0, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
            tmem_st32(t_lane + kKv4TmemO + c0, x);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        mo = fmaxf(mo, m);
        uint4* w = reinterpret_cast<uint4*>((from_peer ? p_peer : p_own) + h * 16);
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {                  // weights move up to the output's
          const float mc = c < 4 ? ma : mb;
          if (!(mc < mo)) continue;
          const float f = fast_exp2(mc - mo);
          uint4 y = w[c * kAttnHeads];
          y.x = scale_bf16x2(y.x, f);
          y.y = scale_bf16x2(y.y, f);
          y.z = scale_bf16x2(y.z, f);
          y.w = scale_bf16x2(y.w, f);
          w[c * kAttnHeads] = y;
        }
        fence_proxy_async_smem();
        warp_arrive(&sm->fix_done);
      }
      if (!ok || !(ok = wait(&sm->fin_own, live) && wait_peer(&sm->fin_peer, live))) break;
      // the output rows are relative to the largest reference; a NaN goes through
      float m = -kInf, l = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, sm->fin[i >> 1][i & 1][1][h]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lp = sm->fin[i >> 1][i & 1][0][h], mp = sm->fin[i >> 1][i & 1][1][h];
        l += lp > 0.f ? lp * fast_exp2(mp - m) : lp;
      }
      __syncwarp();
      if (h == 0) mbar_arrive_expect_tx(&sm->fin_peer, kFinBytes);
      if (lane == 0) {
        mbar_arrive(&sm->fin_free);
        mbar_arrive_remote(peer_fin_free);
      }
      tc_fence_after();
      const float inv = l != 0.f ? 1.f / l : 0.f;      // every logit -inf: as an empty set
#pragma unroll 1
      for (int c0 = 0; c0 < 256; c0 += 32) {
        uint32_t x[32];
        tmem_ld32(t_lane + kKv4TmemO + c0, x);
        tmem_wait_ld();
        if (c0 == 224) {                               // all of it is in registers
          tc_fence_before();
          warp_arrive(&sm->o_empty);
        }
        if (!head_ok) continue;
        if (p.parts > 1) {
          float4* dst = reinterpret_cast<float4*>(p.part_o + (orow * p.parts + it.part) * kAttnDv + rank * 256 + c0);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(x[4 * i]) * inv, __uint_as_float(x[4 * i + 1]) * inv,
                                 __uint_as_float(x[4 * i + 2]) * inv, __uint_as_float(x[4 * i + 3]) * inv);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              w[q] = pack_bf16x2(__uint_as_float(x[16 * i + 2 * q]) * inv, __uint_as_float(x[16 * i + 2 * q + 1]) * inv);
            stg256(out + c0 + 16 * i, w);
          }
        }
      }
      if (rank == 0 && head_ok) {
        const float x = (m + log2f(l)) * 0.69314718055994531f;
        if (p.parts > 1) p.part_lse[orow * p.parts + it.part] = x;
        else p.lse[p.row0 * p.heads + orow] = x;
      }
      ++live;
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
// without keys has lse_i = -inf, weight 0 and no output to read; a part whose
// lse is NaN makes o and lse NaN, also where no other part has keys (fmaxf
// leaves it out of the maximum, which is then -inf).  Eight parts' loads are in
// flight at a time.
constexpr int kKv4MaxParts = kKv4MaxK / kAttnTileN;
__global__ void __launch_bounds__(128) kv4_join_kernel(const Kv4AttnParams p) {
  __shared__ float weight[kKv4MaxParts];
  const int64_t orow = blockIdx.x, out = p.row0 * p.heads + orow;
  const float kInf = __int_as_float(0x7f800000);
  const float* pl = p.part_lse + orow * p.parts;
  const float* po = p.part_o + orow * p.parts * kAttnDv + threadIdx.x * 4;
  const int lane = threadIdx.x & 31;
  wait_for_previous_kernel();
  float top = -kInf;
  for (int i = lane; i < p.parts; i += 32) top = fmaxf(top, pl[i]);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
  float z = 0.f;
  for (int i = lane; i < p.parts; i += 32) {
    const float w = pl[i] == -kInf ? 0.f : expf(pl[i] - top);
    z += w;
    if (threadIdx.x < 32) weight[i] = w;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) z += __shfl_xor_sync(kFull, z, o);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < p.parts; i0 += 8) {
    float4 v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      v[u] = i0 + u < p.parts && weight[i0 + u] != 0.f ? *reinterpret_cast<const float4*>(po + static_cast<int64_t>(i0 + u) * kAttnDv)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float w = i0 + u < p.parts ? weight[i0 + u] : 0.f;
      acc.x += w * v[u].x; acc.y += w * v[u].y; acc.z += w * v[u].z; acc.w += w * v[u].w;
    }
  }
  const float inv = z > 0.f ? 1.f / z : z;               // no key at all: 0; a NaN goes through
  *reinterpret_cast<uint2*>(p.o + out * kAttnDv + threadIdx.x * 4) =
      make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (threadIdx.x == 0) p.lse[out] = top + logf(z);    // -inf + log 0 = -inf for an empty set
}

}  // namespace hisa
