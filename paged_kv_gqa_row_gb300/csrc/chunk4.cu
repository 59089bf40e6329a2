// K4 over 4-bit pools (LNK_KV_E2M1): packed prompt chunks on the fifth-generation
// tensor cores, two SMs per tile.
//
// The tiles, their runs of steps and the two products of a step are chunk.cu's
// (256 query rows of one kv head per cluster of two CTAs, 128 keys a step, S and P
// in tensor memory).  Three things differ.
//
// The operands.  The tensor cores read f16 tiles that this kernel makes from the
// packed pages: a code times its block's scale is exact in f16 (at most five
// significant bits, 2^-10 .. 2688); queries (exact in the range the header states)
// and P are f16 too, as both operands of a product have one type.  P is relative to
// 2^-7 of the row's reference, which the largest score may exceed by 2^8 before the
// reference follows: at most 2^15 in f16, rounded to 2^-11 relative down to 2^-21 of
// the reference, and what smaller ones lose is below 2^-32 of it each.  (The factor
// is in the sums too.)
//
// The tiles follow one another without a pause.  One cluster per pair of SMs takes
// its share of the (tile, kv head) items in turn, and every ring and barrier runs
// on over their ends, counted by the steps of all of the cluster's tiles (J below):
// while the softmax ends a tile, the next one's runs are known, its first pages
// are converted and its queries loaded.
//
// And the code is short.  Softmax and converting warps share the schedulers, and
// with a softmax written out for the 128 scores of a step (as chunk.cu has it, where
// nothing else runs beside it) warps waited for instructions more than for anything
// else.  So the scores stay in tensor memory and are read twice, in loops of 64 (for
// the maximum) and 32 (for P): the example below took 223 us with the written-out
// softmax, 177 us with 64 scores at a time throughout, 164 us with 32.
//
// Tensor memory holds three score buffers and O.  P takes the place of the scores it
// is made from, in two halves, so that P.V starts on the first while the softmax
// writes the second.
//
// What bounds it: the chain of one step, products of 500 cycles each behind one
// another, a softmax of 2500 cycles, three steps in flight; the tensor cores are busy a
// third of the time.  Four prompts of 1024 to 2047 tokens, 32 query heads on 8,
// D = 128: 129 us, 637 TFLOP/s (chunk.cu on bf16 pools 181 us).  Four prompts of 512
// tokens after 1024 to 7168 others, with 32 decode rows: 190 us (bf16 pools 255 us).
// Eight converting warps instead of four (fewer registers for all) took 10% longer,
// deeper rings of tiles and shallower ones of packed pages as long; the next tile's
// first step before a tile's end, or one loop for the keys' and the values'
// conversion, 4 to 10% longer.
//
// CTA structure (512 threads in both ranks):
//  * warp 0, producer: this CTA's K page and both V pages of a step as they are
//    (36 D bytes each, 1-D bulk copies) into a ring of packed stages, with a
//    record of the step (its real keys, first key, run);
//  * warp 1: in rank 0 the Q.K^T issuer; in rank 1 the keys' relay;
//  * warp 2: in rank 0 the P.V issuer; in rank 1 the values' relay;
//  * warp 3, set-up: finds the tokens and runs of the tiles ahead (two slots);
//  * warps 4-11, softmax: two groups of four warps that take the steps in turn;
//    thread r of a group owns query row r of its CTA (tensor-memory lane r);
//  * warps 12-15 convert: a thread takes 16 dimensions of one key (8 code bytes
//    and their scale) and stores them as two 16-byte pieces of the swizzled tile,
//    zeros for the value rows outside the real keys.  They also load the queries
//    of the next tile beside those of the tile before.  They arrive on barriers of
//    their own CTA, and the relays pass that on to rank 0: the arrival that
//    publishes stores to the other CTA takes 600 to 900 cycles, and made by the
//    converting warps themselves it doubled the time of a step.
//
// NaN.  A product multiplies every value row of a step into all 256 query rows, and
// P = 0 does not keep a NaN out.  So value blocks with a NaN scale are converted as
// finite numbers, and a converting thread that meets one notes the tile in both CTAs.
// At the end of such a tile each softmax thread looks through the scales of the keys
// that its row sees, and the 16 dimensions of a NaN block become NaN in its output.
// (Keys need nothing: the scores that a row does not see are replaced.)
//
// Sources: as chunk.cu; the 4-bit format is this library's (lnk_attn_desc).
#include <map>
#include <mutex>
#include <type_traits>
#include <utility>

#include "common.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

constexpr int kThreads = 16 * 32;
constexpr int kPvWarp = 2, kSetupWarp = 3, kSoftmaxWarp = 4, kConvertWarp = 12;
constexpr int kConvertThreads = 128;
constexpr int kStagesK = 3;               // K ring (this CTA's page of a step)
constexpr int kStagesV = 3;               // V ring (this CTA's columns of both pages)
constexpr int kStagesP = 3;               // packed stages
constexpr int kScores = 3;                // score buffers in tensor memory
constexpr int kRows = 128;                // query rows per CTA = tensor-memory lanes
constexpr int kTileRows = 2 * kRows;      // rows of a tile (both CTAs)
constexpr int kStepKeys = 2 * kPage;      // keys per step
constexpr float kRescaleLog2 = 8.f;       // rescale O when the max grows by more than 2^8
constexpr float kHeadroomLog2 = 7.f;      // a score at the reference has P = 2^7 (f16 ends at 65504)
constexpr int kMaxOrderedTiles = 512;     // tiles ordered by cost (larger launches keep token order)
// Step records that the producer writes and the converting and the softmax warps
// read.  Step J is recorded once step J - 3 is converted, so after
// Q.K^T of step J - 6, for which P of step J - 9 was written and read: 16 are enough.
constexpr int kStepRecords = 16;

// A tile of the cluster's, as the set-up warp leaves it for the others.
struct Tile {
  int t0, nt, h, steps, nruns;
  int lo[kTileRows], hi[kTileRows], run[kTileRows];       // per token: visible keys [lo, hi), its run (-1: none)
  int row[kTileRows], kmin[kTileRows], kmax[kTileRows];  // per run: table row, keys [kmin, kmax)
};
// Notes of NaN value blocks, of tile n in place n mod kNanNotes.  A converting warp at
// tile n + 4 has found the queries of n + 2 done with in its own CTA, whose softmax
// came after P.V of n + 2, so after O of n + 1 was read in both CTAs: none of them
// still asks for tile n.
constexpr int kNanNotes = 4;
constexpr int kTileReaders = 15;  // producer, warps 1 and 2, eight softmax and four converting warps

template <int D>
struct Smem {
  static constexpr int kPageBytes = 36 * D;                 // a packed page
  static constexpr int NB = boxes_for(D);
  static constexpr int kKStage = NB * kBoxBytes;            // one page of K, all head-dim columns
  static constexpr int kVStage = 2 * kBoxBytes;             // both pages of V, 64 head-dim columns
  static constexpr int kPvN = 128;                          // N of P.V (head_dim padded; 64 per CTA)
  static constexpr uint32_t kTmemCols = 512;
  // tensor-memory columns: S_0, S_1, S_2 (f32 scores; P_b, f16 pairs, takes the
  // first half of S_b as the softmax reads it), O
  static constexpr uint32_t kColS = 0, kColO = kScores * kStepKeys;
  static_assert(kColO + kPvN <= kTmemCols, "tensor memory");
  static constexpr int kQBox = kRows * 128;                 // 128 query rows x 64 head-dim columns
  static constexpr size_t kring = 0;
  static constexpr size_t vring = kring + size_t(kStagesK) * kKStage;
  static constexpr size_t qsm = vring + size_t(kStagesV) * kVStage;  // this CTA's query rows, K-major
  static constexpr int kQTile = NB * kQBox;                 // two of them, for two tiles in turn
  static constexpr size_t packed = qsm + size_t(2) * kQTile;  // [kStagesP]: K page, V page a, V page b
  static constexpr size_t bars = packed + size_t(kStagesP) * 3 * kPageBytes;
  // kfull[K], kempty[K], vfull[V], vempty[V], rawfull[P], rawempty[P], sfull[3], pfull[6], pvdone[3], tfull[2],
  // tempty[2], odone, ofree, qfull[2], qempty[2]
  static constexpr int kNumBars = 2 * (kStagesK + kStagesV + kStagesP) + 4 * kScores + 10;
  static constexpr size_t records = (bars + kNumBars * sizeof(uint64_t) + 15) / 16 * 16;  // [kStepRecords] int4
  static constexpr size_t tiles = records + size_t(kStepRecords) * 16;  // [2] Tile
  static constexpr size_t misc = tiles + 2 * sizeof(Tile);              // abort, tensor-memory address
  static constexpr size_t nans = misc + 16;                             // [kNanNotes]: last tile noted, plus one
  static constexpr size_t order = nans + kNanNotes * 4;                            // [kMaxOrderedTiles]: uint16 tiles by cost
  // softmax groups' hand-off: max [2][128] and ok [2][128] per step parity; at a
  // tile's end max, sum and ok [2][128] per group and tile parity.  Before the
  // first tile: the tiles' costs.
  static constexpr size_t xchg = order + kMaxOrderedTiles * 2;
  static constexpr size_t end = xchg + 16 * kRows * 4;
  static constexpr size_t bytes = end + 1024;
  static_assert(kMaxOrderedTiles * 4 <= 16 * kRows * 4, "the costs fit the hand-off");
  static_assert(bytes <= 227 * 1024, "one CTA's shared memory");
};

// The cluster's k-th item of all (tile, kv head) items in the order of cost: rounds
// of one item per cluster, every other one backwards, so that the sums even out.
// Items past the end come last, in every cluster.
__device__ __forceinline__ long long item_of(int k, int clusters, int cluster) {
  return static_cast<long long>(k) * clusters + ((k & 1) ? clusters - 1 - cluster : cluster);
}

// 128 threads: a tile's query rows of this CTA into shared memory as f16 (K-major,
// 128-byte swizzle: the A operand of Q.K^T), a thread per row: its 16-byte pieces
// are loaded before any is stored.  The caller publishes them to the pair's tensor
// cores (each thread orders its stores before the async proxy here).
template <int D>
__device__ __forceinline__ void load_queries(const ChunkParams& p, uint8_t* q, int t0, int h, uint32_t rank, int rl) {
  const int row = static_cast<int>(rank) * kRows + rl;  // token * G + head
  const int tl = row / p.group, g = row % p.group;
  const bool real = tl < min(2 * p.tile_tokens, p.P - t0);
  const uint4* src = reinterpret_cast<const uint4*>(
      p.q + (real ? (static_cast<size_t>(t0 + tl) * p.hq + static_cast<size_t>(h) * p.group + g) * D : 0));
  uint4 a[D / 8];
#pragma unroll
  for (int c = 0; c < D / 8; ++c) a[c] = real ? src[c] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int c = 0; c < D / 8; ++c)
    *reinterpret_cast<uint4*>(q + (c >> 3) * (kRows * 128) + swz128(rl, c & 7)) =
        make_uint4(bf16x2_to_f16x2(a[c].x), bf16x2_to_f16x2(a[c].y), bf16x2_to_f16x2(a[c].z), bf16x2_to_f16x2(a[c].w));
  fence_proxy_async_smem();
}

constexpr int kPastRun = -2147483647 - 1;  // "entry" of a page past the end of its run

// Walks a tile's steps in order: the run's pages page, page + 1, the second one
// past the run's last page when the run has an odd number of pages.
struct Walk {
  int run = -1, page = 0, last = -1, kmin = 0, kmax = 0;
  const int* trow = nullptr;
  __device__ __forceinline__ void next(const ChunkParams& p, const Tile& t) {
    page += 2;
    if (page <= last) return;
    if (++run >= t.nruns) return;
    kmin = t.kmin[run];
    kmax = t.kmax[run];
    page = kmin / kPage;
    last = (kmax - 1) / kPage;
    trow = p.table + static_cast<long long>(t.row[run]) * p.pages_per_row;
  }
  // Table entries of the step's two pages (kPastRun for a page past its run, and
  // for both past the last run).
  __device__ __forceinline__ void entries(const Tile& t, int& ea, int& eb) const {
    ea = eb = kPastRun;
    if (run >= t.nruns) return;
    ea = trow[page];
    if (page < last) eb = trow[page + 1];
  }
};

// One warp: the tokens and runs of the tile at `item`.  Runs are maximal groups of
// the tile's valid tokens (in order, skipping tokens that see no key) with one
// table row.
__device__ __forceinline__ void set_up(const ChunkParams& p, Tile& t, int tile, int h, uint32_t rank, int lane) {
  const int TQ = 2 * p.tile_tokens;
  const int t0 = tile * TQ;
  const int nt = min(TQ, p.P - t0);
  int nr = 0;           // runs so far
  int last_row = 0;     // row of the last valid token so far
  bool have_last = false;
  int npos = lane < nt ? p.positions[t0 + lane] : -1;  // the next 32 tokens, read ahead
  int nrow = lane < nt ? p.rows[t0 + lane] : -1;
  for (int base = 0; base < TQ; base += 32) {
    const int i = base + lane;
    const int pos = npos, row = nrow;
    npos = i + 32 < nt ? p.positions[t0 + i + 32] : -1;
    nrow = i + 32 < nt ? p.rows[t0 + i + 32] : -1;
    int lo = 0, hi = 0, bad = 0;
    if (pos >= 0) {
      if (row < 0 || row >= p.num_rows) bad = LNK_DEV_BAD_ROW;
      else if (pos >= p.pages_per_row * kPage) bad = LNK_DEV_BAD_POSITION;
      else {
        lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        hi = pos + 1;
      }
    }
    if (h == 0 && rank == 0 && p.status != nullptr) {
      if (p.segments != nullptr && i < nt && t0 + i > 0 && p.segments[t0 + i] == p.segments[t0 + i - 1] &&
          row != p.rows[t0 + i - 1])
        bad |= LNK_DEV_SEGMENT;
      if (bad) atomicOr(p.status, bad);
    }
    const bool v = hi > lo;
    const unsigned vm = __ballot_sync(0xffffffffu, v);
    // row of the previous valid token: in this group of 32, else carried over
    const unsigned before = vm & ((1u << lane) - 1u);
    const int prev = __shfl_sync(0xffffffffu, row, before ? 31 - __clz(before) : lane);
    const bool has_prev = before != 0u || have_last;
    const int prev_row = before ? prev : last_row;
    const bool start = v && (!has_prev || prev_row != row);
    const unsigned sm = __ballot_sync(0xffffffffu, start);
    const int rid = nr + __popc(sm & ((2u << lane) - 1u)) - 1;  // (lane 31: all bits)
    if (i < TQ) {
      t.lo[i] = lo;
      t.hi[i] = hi;
      t.run[i] = v ? rid : -1;
    }
    if (start) {
      t.row[rid] = row;
      t.kmin[rid] = lo;
      t.kmax[rid] = hi;
    }
    __syncwarp();
    if (v && !start) {
      atomicMin(t.kmin + rid, lo);
      atomicMax(t.kmax + rid, hi);
    }
    __syncwarp();
    nr += __popc(sm);
    if (vm) {
      last_row = __shfl_sync(0xffffffffu, row, 31 - __clz(vm));
      have_last = true;
    }
  }
  int steps = 0;
  for (int r = lane; r < nr; r += 32) steps += ((t.kmax[r] - 1) / kPage - t.kmin[r] / kPage + 2) / 2;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) steps += __shfl_xor_sync(0xffffffffu, steps, o);
  if (lane == 0) {
    t.t0 = t0;
    t.nt = nt;
    t.h = h;
    t.steps = steps;
    t.nruns = nr;
  }
  __syncwarp();
}

// A word of shared memory of this CTA or the peer (mapa_shared).
__device__ __forceinline__ void store_cluster(uint32_t cluster_addr, int value) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(value) : "memory");
}

__device__ __forceinline__ uint32_t max_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One 64-column box of a packed page for the converting warps: NBLK of the row's
// blocks, from b0; thread t takes block b0 + t % NBLK of rows t / NBLK, + kAtOnce,
// ...  Loads and stores are apart, so that the loads of several boxes are in
// flight before the first store.
template <int D, int NBLK>
struct Box {
  static constexpr int kAtOnce = kConvertThreads / NBLK;  // rows
  static constexpr int kUnits = kAtOnce >= kPage ? 1 : kPage / kAtOnce;
  static_assert(kPage % kAtOnce == 0, "whole passes");
  uint2 w[kUnits];     // 16 codes
  uint32_t s[kUnits];  // their scale

  __device__ __forceinline__ void load(const uint8_t* src, int b0, int t) {
    const int b = b0 + t % NBLK;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int j = u * kAtOnce + t / NBLK;
      w[u] = *reinterpret_cast<const uint2*>(src + j * (D / 2) + b * 8);
      s[u] = src[32 * D + ((j & 3) * (D / 16) + b) * 16 + (j >> 2)];
    }
  }
  // Into the swizzled f16 tile `dst`; rows outside [x, y) get zeros.  FINITE: a NaN
  // scale becomes the least finite one (a maximum drops the NaN), and the result is
  // not zero if there was one.
  template <bool FINITE>
  __device__ __forceinline__ uint32_t store(uint8_t* dst, int t, int x, int y) const {
    const int lb = t % NBLK;
    uint32_t dropped = 0u;
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int j = u * kAtOnce + t / NBLK;
      const uint32_t sc = j < x || j >= y ? 0u : s[u];  // (codes are finite: zero)
      uint32_t s2 = e4m3x2_to_f16x2(sc | (sc << 8));
      if constexpr (FINITE) {
        const uint32_t f2 = max_f16x2(s2, 0xDF00DF00u);  // (-448, twice)
        dropped |= s2 ^ f2;
        s2 = f2;
      }
      uint32_t lo[4], hi[4];
      e2m1x8_to_f16x2x4(w[u].x, lo);
      e2m1x8_to_f16x2x4(w[u].y, hi);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] = mul_f16x2(lo[i], s2);
        hi[i] = mul_f16x2(hi[i], s2);
      }
      *reinterpret_cast<uint4*>(dst + swz128(j, 2 * lb)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(dst + swz128(j, 2 * lb + 1)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
    return dropped;
  }
};

// The blocks b0 .. b0 + D/32 - 1 (as bits from 0) with a NaN scale in any of the values
// at positions [lo, hi) of a table row, one kv head's pages at `pool`.
template <int D>
__device__ __noinline__ uint32_t nan_blocks(const uint8_t* pool, const int32_t* trow, int num_pages, int lo, int hi, int b0) {
  uint32_t blocks = 0u;
#pragma unroll 1
  for (int lp = lo / kPage; lp <= (hi - 1) / kPage; ++lp) {
    const int page = trow[lp];
    if (page < 0 || page >= num_pages) continue;
    const uint8_t* scales = pool + static_cast<size_t>(page) * (36 * D) + 32 * D;
#pragma unroll 1
    for (int i = 0; i < 4 * (D / 32); ++i) {  // positions q, q + 4, ... of a page, one block
      const int q = i & 3, b = i >> 2;
      const uint4 x = *reinterpret_cast<const uint4*>(scales + (q * (D / 16) + b0 + b) * 16);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int y = 0; y < 16; ++y) {
        const int j = lp * kPage + q + 4 * y;
        if (((w[y >> 2] >> (8 * (y & 3))) & 0x7Fu) == 0x7Fu && j >= lo && j < hi) blocks |= 1u << b;
      }
    }
  }
  return blocks;
}

constexpr int kPass = 32;  // scores of a row that P is made of at once (the maximum: twice as many)

template <int N>
__device__ __forceinline__ void load_scores(uint32_t col, float (&x)[N]) {
#pragma unroll
  for (int h = 0; h < N / 32; ++h) {
    uint32_t (&r)[32] = *reinterpret_cast<uint32_t(*)[32]>(x + 32 * h);
    tmem_ld32(col + 32 * h, r);
  }
  tmem_ld_wait();
}

// Scores outside [a, e) become -inf.
template <int N>
__device__ __forceinline__ void mask_scores(float (&x)[N], int a, int e) {
#pragma unroll
  for (int h = 0; h < N / 32; ++h) {
    const int first = min(max(a - 32 * h, 0), 32), end = min(max(e - 32 * h, 0), 32);
    const uint32_t in = end <= first ? 0u : (0xffffffffu >> (32 - (end - first))) << first;
#pragma unroll
    for (int i = 0; i < 32; ++i) x[32 * h + i] = (in >> i) & 1u ? x[32 * h + i] : -INFINITY;
  }
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) chunk4_kernel(const ChunkParams p) {
  using L = Smem<D>;
  constexpr int DK = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* kempty = kfull + kStagesK;
  uint64_t* vfull = kempty + kStagesK;
  uint64_t* vempty = vfull + kStagesV;
  uint64_t* rawfull = vempty + kStagesV;  // packed stages
  uint64_t* rawempty = rawfull + kStagesP;
  uint64_t* sfull = rawempty + kStagesP;  // [kScores] Q.K^T into S_b finished
  uint64_t* pfull = sfull + kScores;      // [kScores][2] a half of P_b written (rank 0 only)
  uint64_t* pvdone = pfull + 2 * kScores;  // [kScores] P.V from P_b finished
  uint64_t* tfull = pvdone + kScores;     // [2] a slot's tile is set up
  uint64_t* tempty = tfull + 2;           // [2] all have read it
  uint64_t* odone = tempty + 2;           // the last P.V of a tile finished
  uint64_t* ofree = odone + 1;            // the softmax has read O (rank 0 only)
  uint64_t* qfull = ofree + 1;            // [2] a tile's queries stored in both CTAs (rank 0 only)
  uint64_t* qempty = qfull + 2;           // [2] the tile's last Q.K^T finished, and its outputs left the buffer
  int4* records = reinterpret_cast<int4*>(smem + L::records);
  Tile* tiles = reinterpret_cast<Tile*>(smem + L::tiles);
  int* misc = reinterpret_cast<int*>(smem + L::misc);
  volatile int* nan_notes = reinterpret_cast<volatile int*>(smem + L::nans);
  uint16_t* order = reinterpret_cast<uint16_t*>(smem + L::order);
  volatile int* abort_flag = misc;

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const uint32_t rank = cluster_cta_rank();
  const int cluster = static_cast<int>(blockIdx.x >> 1), clusters = static_cast<int>(gridDim.x >> 1);
  const int G = p.group;
  const int TQ = 2 * p.tile_tokens;  // tokens of a tile
  const long long items = static_cast<long long>(p.num_tiles) * p.hkv;
  const bool ordered = items > clusters && p.num_tiles <= kMaxOrderedTiles;  // (one round needs no order)

  if (tid == 0) {
    // rank 0's full barriers also count the relay's arrival for rank 1's tile
    const int nfull = kConvertThreads / 32 + (rank == 0 ? 1 : 0);
    for (int s = 0; s < kStagesK; ++s) {
      mbar_init(smem_addr(kfull + s), nfull);
      mbar_init(smem_addr(kempty + s), 1);
    }
    for (int s = 0; s < kStagesV; ++s) {
      mbar_init(smem_addr(vfull + s), nfull);
      mbar_init(smem_addr(vempty + s), 1);
    }
    for (int s = 0; s < kStagesP; ++s) {
      mbar_init(smem_addr(rawfull + s), 1);
      mbar_init(smem_addr(rawempty + s), kConvertThreads / 32);
    }
    for (int b = 0; b < kScores; ++b) {
      mbar_init(smem_addr(sfull + b), 1);
      mbar_init(smem_addr(pfull + 2 * b), 8);  // one softmax group (four warps) in each CTA
      mbar_init(smem_addr(pfull + 2 * b + 1), 8);
      mbar_init(smem_addr(pvdone + b), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_addr(tfull + b), 1);
      mbar_init(smem_addr(tempty + b), kTileReaders);
      mbar_init(smem_addr(qfull + b), 2 * (kConvertThreads / 32));
      mbar_init(smem_addr(qempty + b), 1 + 8);  // the last Q.K^T, and the softmax warps at the tile's end
    }
    mbar_init(smem_addr(odone), 1);
    mbar_init(smem_addr(ofree), 16);  // both groups in both CTAs
    misc[0] = 0;
    for (int i = 0; i < kNanNotes; ++i) nan_notes[i] = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) tmem2_alloc(smem_addr(misc + 1), L::kTmemCols);
  // (nothing of the caller's is read or written before the previous kernel's end)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // ---- the tiles by estimated cost (pages that its last position sees), longest
  // first; every CTA computes the same order ----
  if (ordered) {
    int* cost = reinterpret_cast<int*>(smem + L::xchg);
    for (int i = tid; i < p.num_tiles; i += kThreads) {
      const int pm = max(p.positions[i * TQ], p.positions[min(p.P, (i + 1) * TQ) - 1]);
      const int pages = pm >= 0 ? pm / kPage + 1 : 0;
      cost[i] = p.window > 0 ? min(pages, (p.window + TQ) / kPage + 2) : pages;
    }
    __syncthreads();
    for (int i = tid; i < p.num_tiles; i += kThreads) {
      const int ci = cost[i];
      int rk = 0;
      for (int k = 0; k < p.num_tiles; ++k) {
        const int ck = cost[k];
        rk += (ck > ci) || (ck == ci && k > i);  // ties: later tokens first
      }
      order[rk] = static_cast<uint16_t>(i);
    }
  }
  __syncthreads();
  auto tile_of = [&](long long item) {
    const int r = static_cast<int>(item / p.hkv);
    return ordered ? static_cast<int>(order[r]) : p.num_tiles - 1 - r;  // (unordered: later tokens first)
  };
  // (every cluster has an item: the launch has at most as many clusters)
  if (warp == kSetupWarp) {
    set_up(p, tiles[0], tile_of(cluster), cluster % p.hkv, rank, lane);
    if (lane == 0) mbar_arrive(smem_addr(tfull));
  } else if (warp >= kSoftmaxWarp && warp < kSoftmaxWarp + 4) {
    // (the cluster barrier below publishes them)
    load_queries<D>(p, smem + L::qsm, tile_of(cluster) * TQ, cluster % p.hkv, rank, tid - kSoftmaxWarp * 32);
  }
  // barriers initialised and tensor memory allocated in both CTAs before any
  // thread of either uses them
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(misc[1]);

  // Each role walks the cluster's tiles k = 0, 1, ... (slot k mod 2) and their steps;
  // J counts the steps of all tiles so far, n the tiles with any step.  A role that
  // gave up a wait leaves its loop: the abort flag makes the others' waits give up.
  auto tile_ready = [&](int k) { return k == 0 || mbar_wait(smem_addr(tfull + (k & 1)), (k >> 1) & 1, abort_flag); };

  if (warp < kSoftmaxWarp) {
    if (warp == 0) {
      // ============================== producer ==============================
      if (lane == 0) {
        int J = 0;
        bool ok = true;
        for (int k = 0; ok && item_of(k, clusters, cluster) < items; ++k) {
          if (!tile_ready(k)) break;
          const Tile& t = tiles[k & 1];
          const int nsteps = t.steps;
          const size_t head = static_cast<size_t>(t.h) * p.num_pages;
          Walk cur;
          int ea, eb;  // table entries of the step's two pages, read one step ahead
          cur.next(p, t);
          cur.entries(t, ea, eb);
          for (int j = 0; j < nsteps; ++j, ++J) {
            const int sp = J % kStagesP;
            Walk nxt = cur;
            int na, nb;
            nxt.next(p, t);
            nxt.entries(t, na, nb);
            // a page past the run or a bad table entry loads page 0 instead (its
            // keys are masked and its values zeroed)
            const bool bad_a = ea >= p.num_pages || ea < 0;
            const bool bad_b = eb != kPastRun && (eb >= p.num_pages || eb < 0);
            if (rank == 0 && (bad_a || bad_b) && p.status != nullptr) atomicOr(p.status, LNK_DEV_BAD_PAGE);
            const int pa = bad_a ? 0 : ea, pb = (bad_b || eb == kPastRun) ? 0 : eb;
            if (J >= kStagesP && !mbar_wait(smem_addr(rawempty + sp), ((J / kStagesP) - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            const int kb = cur.page * kPage;
            records[J % kStepRecords] =
                make_int4(max(cur.kmin - kb, bad_a ? kPage : 0),
                          min(cur.kmax - kb, (bad_b || eb == kPastRun) ? kPage : kStepKeys), kb, cur.run);
            const uint32_t fb = smem_addr(rawfull + sp);
            mbar_arrive_expect_tx(fb, 3 * L::kPageBytes);
            const uint32_t dst = smem_addr(smem + L::packed + size_t(sp) * 3 * L::kPageBytes);
            bulk_load(dst, p.k_pool + (head + (rank == 0 ? pa : pb)) * L::kPageBytes, L::kPageBytes, fb);
            bulk_load(dst + L::kPageBytes, p.v_pool + (head + pa) * L::kPageBytes, L::kPageBytes, fb);
            bulk_load(dst + 2 * L::kPageBytes, p.v_pool + (head + pb) * L::kPageBytes, L::kPageBytes, fb);
            cur = nxt;
            ea = na;
            eb = nb;
          }
          mbar_arrive(smem_addr(tempty + (k & 1)));
        }
        // do not leave while a copy may still land in this CTA's memory
        for (int kk = max(0, J - kStagesP); kk < J; ++kk) {
          const uint32_t fb = smem_addr(rawfull + kk % kStagesP);
          const uint64_t t_0 = global_timer_ns();
          while (!mbar_try_wait(fb, (kk / kStagesP) & 1) && global_timer_ns() - t_0 < kWaitLimitNs) {
          }
        }
      }
    } else if (warp == 1 || warp == kPvWarp) {
      if (lane == 0 && rank != 0) {
        // ============================ relays (rank 1) =========================
        // publish what this CTA's warps converted: warp 1 keys, warp 2 values
        static_assert(kStagesK == kStagesV, "one loop for both rings");
        uint64_t* full = warp == 1 ? kfull : vfull;
        const uint32_t full0 = mapa_shared(smem_addr(full), 0);
        int J = 0;
        bool ok = true;
        for (int k = 0; ok && item_of(k, clusters, cluster) < items; ++k) {
          if (!tile_ready(k)) break;
          const int nsteps = tiles[k & 1].steps;
          mbar_arrive(smem_addr(tempty + (k & 1)));
          for (int j = 0; j < nsteps; ++j, ++J) {
            ok = mbar_wait(smem_addr(full + J % kStagesK), (J / kStagesK) & 1, abort_flag);
            if (!ok) break;
            mbar_arrive_cluster(full0 + (J % kStagesK) * 8);
          }
        }
      } else if (lane == 0 && warp == 1) {
        // ======================= Q.K^T issuer (rank 0) ========================
        constexpr uint32_t kIdS = umma_idesc_f16(kTileRows, kStepKeys, 0, 0);
        // Descriptors of stage 0's K tile and of the query rows (K-major); another
        // stage or K step adds its byte offset / 16 to the 14-bit address field,
        // which cannot carry (shared addresses stay below 256 KiB).
        const uint64_t kdesc0 = umma_desc_sw128(smem_addr(smem + L::kring), 0, 1024);
        const uint64_t qdesc0 = umma_desc_sw128(smem_addr(smem + L::qsm), 0, 1024);
        // S_b = Q K^T of step J (b = J mod 3), once P.V of step J - 3 has read P_b,
        // both CTAs' K pages are converted and, for the first step of a tile, its
        // queries stored in both CTAs.
        int J = 0, n = 0;
        bool ok = true;
        for (int k = 0; ok && item_of(k, clusters, cluster) < items; ++k) {
          if (!tile_ready(k)) break;
          const int nsteps = tiles[k & 1].steps;
          mbar_arrive(smem_addr(tempty + (k & 1)));
          if (nsteps == 0) continue;
          ok = mbar_wait_cluster(smem_addr(qfull + (n & 1)), (n >> 1) & 1, abort_flag);
          const uint64_t qd = qdesc0 + static_cast<uint64_t>(((n & 1) * L::kQTile) >> 4);
          for (int j = 0; ok && j < nsteps; ++j, ++J) {
            const int b = J % kScores, sk = J % kStagesK;
            ok = (J < kScores || mbar_wait(smem_addr(pvdone + b), (J / kScores - 1) & 1, abort_flag)) &&
                 mbar_wait_cluster(smem_addr(kfull + sk), (J / kStagesK) & 1, abort_flag);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sc = tmem + L::kColS + static_cast<uint32_t>(b) * kStepKeys;
            const uint64_t kd = kdesc0 + static_cast<uint64_t>((sk * L::kKStage) >> 4);
#pragma unroll
            for (int kk = 0; kk < DK; ++kk) {
              const uint32_t koff = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
              const uint32_t qoff = ((kk >> 2) * L::kQBox + (kk & 3) * 32) >> 4;
              umma2_ss(sc, qd + qoff, kd + koff, kIdS, kk > 0);
            }
            umma2_commit_both(smem_addr(sfull + b));
            umma2_commit_both(smem_addr(kempty + sk));
            if (j + 1 == nsteps) umma2_commit_both(smem_addr(qempty + (n & 1)));
          }
          ++n;
        }
      } else if (lane == 0) {
        // ========================= P.V issuer (rank 0) ========================
        // One thread issues every P.V, in step order: O accumulates in order,
        // and a finished P.V implies that every earlier one has finished.  A
        // tile's first P.V overwrites O, once the softmax has read the last one.
        constexpr uint32_t kIdPV = umma_idesc_f16(kTileRows, L::kPvN, 0, 1);
        const uint64_t vdesc0 = umma_desc_sw128(smem_addr(smem + L::vring), 0, 1024);
        int J = 0, n = 0;
        bool ok = true;
        for (int k = 0; ok && item_of(k, clusters, cluster) < items; ++k) {
          if (!tile_ready(k)) break;
          const int nsteps = tiles[k & 1].steps;
          mbar_arrive(smem_addr(tempty + (k & 1)));
          if (nsteps == 0) continue;
          if (n > 0) ok = mbar_wait(smem_addr(ofree), (n - 1) & 1, abort_flag);
          ++n;
          for (int j = 0; ok && j < nsteps; ++j, ++J) {
            const int b = J % kScores, sv = J % kStagesV;
            ok = mbar_wait_cluster(smem_addr(vfull + sv), (J / kStagesV) & 1, abort_flag);
            const uint32_t pc = tmem + L::kColS + static_cast<uint32_t>(b) * kStepKeys;
            const uint64_t vd = vdesc0 + static_cast<uint64_t>((sv * L::kVStage) >> 4);
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
              ok = ok && mbar_wait(smem_addr(pfull + 2 * b + half), (J / kScores) & 1, abort_flag);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kPage / 16; ++kk) {  // 16 keys per product
                const uint64_t bd = vd + (((half * kPage + kk * 16) * 128) >> 4);
                umma2_ts(tmem + L::kColO, pc + half * (kPage / 2) + kk * 8, bd, kIdPV, (j > 0 || half > 0 || kk > 0));
              }
            }
            if (!ok) break;
            umma2_commit_both(smem_addr(vempty + sv));
            umma2_commit_both(smem_addr(pvdone + b));
            if (j + 1 == nsteps) umma2_commit_both(smem_addr(odone));
          }
        }
      }
    } else {
      // =============================== set-up ===============================
      // (a slot is free when all have read its tile, the producer last)
      for (int k = 1; item_of(k, clusters, cluster) < items; ++k) {
        if (k >= 2 &&
            !__all_sync(0xffffffffu, mbar_wait(smem_addr(tempty + (k & 1)), ((k >> 1) - 1) & 1, abort_flag)))
          break;
        const long long item = item_of(k, clusters, cluster);
        set_up(p, tiles[k & 1], tile_of(item), static_cast<int>(item % p.hkv), rank, lane);
        if (lane == 0) mbar_arrive(smem_addr(tfull + (k & 1)));
      }
    }
  } else if (warp >= kConvertWarp) {
    // ============================= conversion =============================
    const int t = tid - kConvertWarp * 32;
    const uint32_t qfull0 = mapa_shared(smem_addr(qfull), 0);
    int J = 0, n = 0;  // n: tiles with steps before this one
    bool ok = true;
    for (int k = 0; ok && item_of(k, clusters, cluster) < items; ++k) {
      if (!__all_sync(0xffffffffu, tile_ready(k))) break;
      const int nsteps = tiles[k & 1].steps, t0 = tiles[k & 1].t0, h = tiles[k & 1].h;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(tempty + (k & 1)));
      if (nsteps > 0) {
        // the tile's queries, beside those of the tile before
        if (n >= 2) ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(qempty + (n & 1)), ((n >> 1) - 1) & 1, abort_flag));
        if (!ok) break;
        if (k > 0) load_queries<D>(p, smem + L::qsm + (n & 1) * L::kQTile, t0, h, rank, t);
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(qfull0 + (n & 1) * 8);
      }
      for (int step = 0; step < nsteps; ++step, ++J) {
        const int j = J, sp = j % kStagesP, sk = j % kStagesK, sv = j % kStagesV;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(rawfull + sp), (j / kStagesP) & 1, abort_flag));
        if (ok && j >= kStagesK)
          ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(kempty + sk), ((j / kStagesK) - 1) & 1, abort_flag));
        if (!ok) break;
        const int4 real = records[j % kStepRecords];
        const uint8_t* raw = smem + L::packed + size_t(sp) * 3 * L::kPageBytes;
        uint8_t* kt = smem + L::kring + size_t(sk) * L::kKStage;
        constexpr int kRest = D > 64 ? D / 16 - 4 : 4;  // blocks past column 64
        const int tv = static_cast<int>(rank) * 4;      // this CTA's first value block
        {
          // this CTA's K page (masked keys' scores are replaced, whatever they are)
          Box<D, 4> lo;
          Box<D, kRest> hi;
          lo.load(raw, 0, t);
          if constexpr (D > 64) hi.load(raw, 4, t);
          lo.template store<false>(kt, t, 0, kPage);
          if constexpr (D > 64) hi.template store<false>(kt + kBoxBytes, t, 0, kPage);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(kfull + sk));
        // this CTA's 64 value columns of both pages (columns past D hold whatever
        // they hold: the output's columns past D are not read)
        uint8_t* vt = smem + L::vring + size_t(sv) * L::kVStage;
        auto values = [&](auto box, bool any) {
          auto box2 = box;
          if (any) {
            box.load(raw + L::kPageBytes, tv, t);
            box2.load(raw + 2 * L::kPageBytes, tv, t);
          }
          // (the packed stage is in registers)
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(rawempty + sp));
          // every warp waits, whether it has values or not: no arrival for a later
          // use of the stage may come before all those of this one
          if (j >= kStagesV)
            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(vempty + sv), ((j / kStagesV) - 1) & 1, abort_flag));
          if (!ok || !any) return;
          const uint32_t dropped = box.template store<true>(vt, t, real.x, real.y) |
                                   box2.template store<true>(vt + kBoxBytes, t, real.x - kPage, real.y - kPage);
          if (dropped != 0u) {  // (published with the values)
            const uint32_t note = smem_addr(smem + L::nans) + static_cast<uint32_t>(n % kNanNotes) * 4;
            store_cluster(mapa_shared(note, 0), n + 1);
            store_cluster(mapa_shared(note, 1), n + 1);
            __threadfence();
          }
        };
        if (kRest == 4 && D > 64) values(Box<D, 4>{}, true);  // (both CTAs' columns are whole)
        else if (rank == 0) values(Box<D, 4>{}, true);
        else values(Box<D, kRest>{}, D > 64);
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(vfull + sv));
      }
      n += nsteps > 0;
    }
  } else {
    // =============================== softmax ==============================
    // Two groups of four warps take the steps in turn, J mod 2, so that one group's
    // loads and maxima overlap the other's exponentials.  Warps w and w + 4 share
    // the tensor-memory lanes of quarter w % 4: thread r of each group owns query
    // row r of this CTA.  Within a tile the row's running max passes from the group of
    // one step to the group of the next through shared memory (a named barrier that
    // the publisher arrives on and the receiver waits on), together with the
    // decision to go on, so a stop reaches both groups and neither waits for the
    // other in vain.  (At a tile's end both meet, and what they exchange there has
    // the next tile's readiness in it, so they go on or stop together.)
    const int grp = (warp - kSoftmaxWarp) >> 2;
    const int qt = warp & 3;              // tensor-memory lane quarter of this warp
    const int rl = qt * 32 + lane;        // row of this CTA = tensor-memory lane
    const int row = static_cast<int>(rank) * kRows + rl;  // row of the tile = token * G + head
    const int gshift = 31 - __clz(G);     // (a group is 1, 2, 4 or 8 heads)
    const int tl = row >> gshift;
    const uint32_t lanes = static_cast<uint32_t>(qt * 32) << 16;
    const int bar_pub = 1 + qt + 4 * grp;        // this group's hand-off to the other group
    const int bar_sub = 1 + qt + 4 * (grp ^ 1);  // the other group's hand-off to this one
    const int bar_fin = 9 + qt;                  // both groups, once at a tile's end
    float* hand_m = reinterpret_cast<float*>(smem + L::xchg);         // [2 step parities][128 rows]
    int* hand_ok = reinterpret_cast<int*>(smem + L::xchg) + 2 * kRows;  // [2][128]
    float* fin = reinterpret_cast<float*>(smem + L::xchg) + 4 * kRows;  // [2 tile parities]: max, sum, ok [2 groups][128]
    const uint32_t pfull0 = mapa_shared(smem_addr(pfull), 0);
    const uint32_t ofree0 = mapa_shared(smem_addr(ofree), 0);
    // Every wait's outcome is made warp-uniform: the tensor-memory loads and
    // stores that follow are warp-collective.
    bool ok = true, stuck = false;
    int J0 = 0, n = 0;  // steps and tiles with steps before this tile
    // A tile as this thread sees it.  Entering one frees its slot.
    int nsteps, t0, nt, h, lo, hi, run_id;
    auto enter = [&](int k) {
      const Tile& t = tiles[k & 1];
      nsteps = t.steps, t0 = t.t0, nt = t.nt, h = t.h;
      lo = hi = 0, run_id = -1;
      if (tl < nt) lo = t.lo[tl], hi = t.hi[tl], run_id = t.run[tl];
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(tempty + (k & 1)));
    };
    enter(0);
    for (int k = 0;; ++k) {
      const bool live = run_id >= 0;
      float m_ref = -INFINITY;   // the row's running max (log2 units) after this group's last step
      float m_part = -INFINITY;  // reference of this group's partial sum
      float l_part = 0.f;        // sum of this group's probabilities, relative to m_part
      for (int j = (J0 & 1) ^ grp; j < nsteps; j += 2) {  // this group's steps of the tile
        const int J = J0 + j, b = J % kScores;
        const uint32_t sc = tmem + lanes + L::kColS + static_cast<uint32_t>(b) * kStepKeys;  // S_b, and P_b
        bool okw = !stuck && __all_sync(0xffffffffu, mbar_wait(smem_addr(sfull + b), (J / kScores) & 1, abort_flag));
        tc_fence_after();
        // visible keys of this step for this row: its own [ka, ke) where they are
        // real (the producer's record, published with the step's scores)
        const int4 real = records[J % kStepRecords];
        const bool in_run = live && real.w == run_id;
        const int ka = in_run ? max(lo - real.z, 0) : kStepKeys;
        const int ke = in_run ? max(ka, min(hi - real.z, kStepKeys)) : kStepKeys;
        const int a0 = max(ka, real.x), e0 = min(ke, real.y);
        const bool masked = !__all_sync(0xffffffffu, a0 == 0 && e0 == kStepKeys);
        // Two passes over the scores, which stay in tensor memory, each a short loop:
        // the maximum, then the probabilities.
        float mraw = -INFINITY;
        if (okw) {
#pragma unroll 1
          for (int c = 0; c < kStepKeys; c += 2 * kPass) {
            float x[2 * kPass];
            load_scores(sc + c, x);
            if (masked) mask_scores(x, a0 - c, e0 - c);
            // a tree of independent three-input maxima
            float m[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              m[i] = x[i];
#pragma unroll
              for (int e = 8; e + 8 < 2 * kPass; e += 16) m[i] = fmax3(m[i], x[e + i], x[e + 8 + i]);
              m[i] = fmaxf(m[i], x[2 * kPass - 8 + i]);
            }
            mraw = fmax3(mraw, fmax3(m[0], m[1], m[2]), fmax3(fmaxf(m[3], m[4]), m[5], fmaxf(m[6], m[7])));
          }
        }
        // in log2 units, less the headroom (all references are: it cancels)
        const float mx = mraw == -INFINITY ? -INFINITY : fmaf(mraw, p.scale_log2, -kHeadroomLog2);
        // the row's running max before this step, from the group of the step before
        if (j > 0) {
          named_barrier_sync(bar_sub, 64);
          m_ref = hand_m[((J - 1) & 1) * kRows + rl];
          okw = okw && hand_ok[((J - 1) & 1) * kRows + rl] != 0;
        }
        ok = __all_sync(0xffffffffu, okw);
        // new running max: it moves only when this step's max exceeds it by
        // more than 2^8, and then O is rescaled
        float m_new = m_ref, alpha = 1.f;
        if (mx != -INFINITY) {
          if (m_ref == -INFINITY) {
            m_new = mx;
          } else if (mx > m_ref + kRescaleLog2) {
            m_new = mx;
            alpha = exp2f(m_ref - mx);
          }
        }
        // hand it on before the exponentials, so the other group can go on
        if (j + 1 < nsteps) {
          hand_m[grp * kRows + rl] = m_new;
          hand_ok[grp * kRows + rl] = ok ? 1 : 0;
          __syncwarp();
          named_barrier_arrive(bar_pub, 64);
        }
        if (!ok) break;
        m_ref = m_new;
        // this group's partial sum follows the row's reference
        if (m_part != m_ref) {
          if (m_part != -INFINITY) l_part *= exp2f(m_part - m_ref);
          m_part = m_ref;
        }
        if (__any_sync(0xffffffffu, alpha != 1.f) && j >= 1) {
          // the running max grew: rescale this row of O once P.V of step J - 1
          // (written by the other group) has finished, before P.V of step J.  (Its
          // parity tells that step from J - 4 only if J - 4 has finished.  P.V runs
          // in step order, so the wait for J - 3, which Q.K^T of step J waited for
          // too, tells that.)
          // (this group's hand-off for step J + 1 has gone out already: if a wait
          // gives up, the failure travels with its next hand-off instead)
          if (J >= kScores)
            stuck = stuck || !__all_sync(0xffffffffu, mbar_wait(smem_addr(pvdone + b), (J / kScores - 1) & 1, abort_flag));
          const int bp = (J - 1) % kScores;
          stuck = stuck || !__all_sync(0xffffffffu, mbar_wait(smem_addr(pvdone + bp), ((J - 1) / kScores) & 1, abort_flag));
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < (stuck ? 0 : L::kPvN / 32); ++c) {
            uint32_t r[32];
            tmem_ld32(tmem + lanes + L::kColO + c * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st32(tmem + lanes + L::kColO + c * 32, r);
          }
        }
        // probabilities 2^(s * scale * log2(e) - m_ref), packed to f16 (paired fp32:
        // one fma and one add per two keys)
        const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t c2 = f32x2(p.scale_log2, p.scale_log2), n2 = f32x2(nbase, nbase);
        uint64_t s2[4] = {0ull, 0ull, 0ull, 0ull};  // running sums, two keys per register
        // (a loop of its own for the steps without masked keys: 2% of the call)
        auto probabilities = [&](auto with_mask) {
#pragma unroll 1
          for (int c = 0; c < kStepKeys; c += kPass) {
            float x[kPass];
            load_scores(sc + c, x);
            if constexpr (decltype(with_mask)::value) mask_scores(x, a0 - c, e0 - c);
#pragma unroll
            for (int hh = 0; hh < kPass / 32; ++hh) {
              uint32_t pk[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float a0v, a1v;
                f32x2_split(fma_f32x2(f32x2(x[hh * 32 + 2 * i], x[hh * 32 + 2 * i + 1]), c2, n2), a0v, a1v);
                const float e0v = ex2_approx(a0v), e1v = ex2_approx(a1v);
                s2[i & 3] = add_f32x2(s2[i & 3], f32x2(e0v, e1v));
                pk[i] = pack_f16x2(e0v, e1v);
              }
              tmem_st16(sc + c / 2 + hh * 16, pk);  // (over scores that were read)
            }
            if ((c + kPass) % kPage == 0) {
              // a half of P is written (and O rescaled): P.V may start on it
              tmem_st_wait();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive_remote(pfull0 + (2 * b + c / kPage) * 8);
            }
          }
        };
        if (masked) probabilities(std::true_type{});
        else probabilities(std::false_type{});
        {
          float u0, u1;
          f32x2_split(add_f32x2(add_f32x2(s2[0], s2[1]), add_f32x2(s2[2], s2[3])), u0, u1);
          l_part += u0 + u1;
        }
      }
      // ---- the tile's end: the groups combine their sums, and each normalises and
      // stores half of head_dim ----
      bool okw = ok && !stuck;
      if (okw && nsteps > 0) okw = __all_sync(0xffffffffu, mbar_wait(smem_addr(odone), n & 1, abort_flag));
      tc_fence_after();
      const bool more = item_of(k + 1, clusters, cluster) < items;
      if (okw && more) okw = __all_sync(0xffffffffu, tile_ready(k + 1));
      float* fin_m = fin + (k & 1) * 6 * kRows;
      float* fin_l = fin_m + 2 * kRows;
      float* fin_ok = fin_l + 2 * kRows;
      fin_m[grp * kRows + rl] = m_part;
      fin_l[grp * kRows + rl] = l_part;
      fin_ok[grp * kRows + rl] = okw ? 1.f : 0.f;
      named_barrier_sync(bar_fin, 64);
      const float mo = fin_m[(grp ^ 1) * kRows + rl], lo_ = fin_l[(grp ^ 1) * kRows + rl];
      ok = __all_sync(0xffffffffu, okw && fin_ok[(grp ^ 1) * kRows + rl] != 0.f);
      // both partial sums relative to the final reference (the larger one)
      const float mf = fmaxf(m_part, mo);
      const float la = m_part == -INFINITY ? 0.f : l_part * exp2f(m_part - mf);
      const float lb = mo == -INFINITY ? 0.f : lo_ * exp2f(mo - mf);
      l_part = grp == 0 ? la + lb : lb + la;
      // This group's half of the rows: from tensor memory to the tile's query buffer,
      // which nobody reads any more (a thread has a row), and from there to memory
      // (neighbouring threads have neighbouring 16 bytes; rows stored by a thread
      // each made a third of the stores' lines).
      constexpr int kPieces = D / 16;  // 16-byte pieces of half a row
      uint8_t* stage = smem + L::qsm + (n & 1) * L::kQTile + (grp * 4 + qt) * (32 * D);
      auto place = [&](int rr, int c) {  // (spread over the banks)
        return rr * D + (kPieces == 6 ? c : c ^ ((rr * kPieces / 8) & (kPieces - 1))) * 16;
      };
      const bool any = ok && nsteps > 0;
      if (any) {
        uint32_t nans = 0u;
        if (nan_notes[n % kNanNotes] == n + 1) {
          if (live)
            nans = nan_blocks<D>(p.v_pool + static_cast<size_t>(h) * p.num_pages * L::kPageBytes,
                                 p.table + static_cast<size_t>(p.rows[t0 + tl]) * p.pages_per_row, p.num_pages, lo, hi,
                                 grp * (D / 32));
          __syncwarp();
        }
        const float inv = live && l_part > 0.f ? p.out_scale / l_part : 0.f;
        const uint32_t oc = tmem + lanes + L::kColO + grp * (D / 2);
#pragma unroll 1
        for (int c = 0; c < kPieces; c += 2) {
          uint32_t r[16];
          tmem_ld16(oc + c * 8, r);
          tmem_ld_wait();
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = live ? pack_bf16x2(__uint_as_float(r[2 * i]) * inv, __uint_as_float(r[2 * i + 1]) * inv) : 0u;
          if ((nans >> (c / 2)) & 1u) {  // (two pieces are a block)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0x7FFF7FFFu;
          }
          *reinterpret_cast<uint4*>(stage + place(lane, c)) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(stage + place(lane, c + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
        }
        // O may take the next tile's values
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(ofree0);
      }
      uint16_t* dst = p.out + (static_cast<size_t>(t0) * p.hq + static_cast<size_t>(h) * G) * D + grp * (D / 2);
#pragma unroll 1
      for (int i = lane; i < kPieces * 32; i += 32) {
        const int rr = i / kPieces, c = i % kPieces;
        const int orow = static_cast<int>(rank) * kRows + qt * 32 + rr, ot = orow >> gshift;
        if (ot < nt)
          *reinterpret_cast<uint4*>(dst + (static_cast<size_t>(ot) * p.hq + (orow & (G - 1))) * D + c * 8) =
              any ? *reinterpret_cast<const uint4*>(stage + place(rr, c)) : make_uint4(0u, 0u, 0u, 0u);
      }
      if (nsteps > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(qempty + (n & 1)));
      }
      J0 += nsteps;
      n += nsteps > 0;
      if (ok && more) enter(k + 1);
      if (!ok || !more) break;
    }
  }
  // The next kernel on the stream may start when every CTA has a thread here, at the
  // latest when its set-up warp has set up the cluster's last tile.  (Allowed at the
  // start, the CTAs of a decode kernel that waits took 1% from the last clusters.)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (*abort_flag && lane == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
  // neither CTA frees its tensor memory or leaves while the pair's products,
  // copies or remote arrivals may still touch it
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem2_dealloc(tmem, L::kTmemCols);
}

// Clusters of the kernel that the current device holds at once, asked for once.
template <int D>
cudaError_t resident_clusters(int* clusters) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  static std::mutex mu;
  static std::map<int, int> done;
  std::lock_guard<std::mutex> lock(mu);
  auto it = done.find(dev);
  if (it != done.end()) {
    *clusters = it->second;
    return cudaSuccess;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Smem<D>::bytes;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  err = cudaOccupancyMaxActiveClusters(clusters, chunk4_kernel<D>, &cfg);
  if (err != cudaSuccess) return err;
  if (*clusters < 1) return cudaErrorInvalidConfiguration;
  done[dev] = *clusters;
  return cudaSuccess;
}

template <int D>
cudaError_t launch_chunk4_t(const ChunkParams& p, cudaStream_t stream) {
  const int bytes = static_cast<int>(Smem<D>::bytes);
  cudaError_t err = set_max_dynamic_smem(reinterpret_cast<const void*>(chunk4_kernel<D>), bytes);
  if (err != cudaSuccess) return err;
  int clusters = 0;
  err = resident_clusters<D>(&clusters);
  if (err != cudaSuccess) return err;
  const long long items = static_cast<long long>(p.num_tiles) * p.hkv;
  if (items < clusters) clusters = static_cast<int>(items);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(bytes);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk4_kernel<D>, p);
}

}  // namespace

cudaError_t launch_chunk4(const ChunkParams& p, int head_dim, cudaStream_t stream) {
  if (p.P == 0) return cudaSuccess;
  switch (head_dim) {
    case 64: return launch_chunk4_t<64>(p, stream);
    case 96: return launch_chunk4_t<96>(p, stream);
    case 128: return launch_chunk4_t<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
