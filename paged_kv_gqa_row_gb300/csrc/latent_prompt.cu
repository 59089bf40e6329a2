// Attention of packed prompts over expanded keys and values: head h of a token has keys
// [k_nope (D), k_rope (R, shared by the heads)] and values of D numbers, which the
// caller computed from the latents; a prompt's queries are the last of its keys and see
// them up to themselves.
//
// A tile is 256 consecutive queries of one prompt and one head, taken by a cluster of two
// CTAs as one 2-SM unit (CTA rank r owns rows 128 r .. + 127 in its tensor-memory lanes);
// the prompt's keys are streamed 128 a step:
//   S[256 x 128]  = Q K_j^T   K_j: rank r holds keys 64 r .. + 63 of the step, D + R
//                             numbers each, K-major;
//   O[256 x 128] += P V_j     P from tensor memory, written over the scores that it is made
//                             from; V_j MN-major: rank r holds value columns 64 r .. + 63 of
//                             all 128 keys.
// A step is a chain: product, softmax, product.  So a cluster has two tiles under way, each with
// its own half of tensor memory (scores and output), its own query rows, rings of keys and
// values, producer, issuer and softmax warps: two workers that share nothing but the pipes, one's
// products running while the other's softmax does, ends of tiles included.  A row belongs to one
// thread from its first key to its stored output.  Its running maximum moves only when it
// grows by more than 2^8, which is when O is rescaled (the scheme of the paged prompt
// kernel, chunk.cu).
//
// Bound: the chain of a step, 3600 cycles of which the two workers' products take 2720.  Four
// prompts of 1024 to 2047 tokens, 32 heads, 0.10 Tflop: 132 us with one tile under way, two score
// buffers and two groups of softmax warps that handed the maximum on; 124 with two workers;
// 112 with the products of P's first half begun before the second is there (its first quarter
// 107.5 to 105 at that stage, three quarters 112, each quarter on its own 114); 105 with sums
// in scalars (pairs of float32 cost the registers' order: 113 to 107) and the registers of the
// loading warps given to the softmax; 103 with votes where reductions ended the waits, 105 now that
// rows are repaired at the end: 0.98 Pflop/s.  Scores in halves of 64 keys, the second of the next
// step before this one's P.V: 5 us more.
//
// Tile ids: prompt n's tiles are base(n) = q_starts[n] / 256 + n onwards, which leaves
// every prompt room for its tiles without a sum over the prompts before it; ids without
// queries end at once.
//
// Values that are not finite, at keys that some rows of a tile see and others do not,
// reach all of them through 0 * NaN: a row whose output is not finite computes it again
// from its own keys, if there is such a value among the tile's keys behind it.  That takes
// long behind long prefixes (a warp's 32 rows behind 60 000 keys 0.34 s), so it is done when
// all the worker's tiles are stored and no role waits for another (repair_rows).  Key rows
// past the tile's last key are zeroed.
#include <algorithm>

#include "latent.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

constexpr int kThreads = 12 * 32;
constexpr int kWorkers = 2;               // tiles that a cluster has under way
constexpr int kStages = 2;                // steps of keys in a worker's ring (of values: one)
constexpr int kRows = 128;                // query rows per CTA = tensor-memory lanes
constexpr int kTileRows = 2 * kRows;
constexpr int kStepKeys = 128;
constexpr float kRescaleLog2 = 8.f;
constexpr int kMaxOrderedTiles = 512;     // tiles ordered by cost (larger launches: later ids first)

template <int D>
struct PromptSmem {
  static constexpr int kBoxesK = D / 64 + 1;                // the last: the rotated numbers
  static constexpr int kKStage = kBoxesK * kBoxBytes;       // this CTA's 64 keys
  static constexpr int kVStage = 2 * kBoxBytes;             // 128 keys, 64 columns
  static constexpr int kQBox = kRows * 128;
  static constexpr int kQ = kBoxesK * kQBox;                // this CTA's 128 query rows
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColS = 0, kColO = 256;         // [worker] 128 columns each; P in the first 64 of S
  // a worker's query rows, keys and values
  static constexpr size_t q = 0;
  static constexpr size_t k = q + kQ;
  static constexpr size_t v = k + size_t(kStages) * kKStage;
  static constexpr size_t worker = v + kVStage;
  // [worker] kfull, kempty [stages], qfull[2], iempty[2], qempty, vfull, vempty, sfull, pfull[2], pvdone, efree
  static constexpr size_t bars = kWorkers * worker;
  static constexpr int kNumBars = 2 * kStages + 12;
  static constexpr size_t misc = bars + kWorkers * kNumBars * sizeof(uint64_t);  // [0] abort, [1] tensor memory, [2] tiles in order, [3] [4] repair
  static constexpr size_t info = misc + 64;                    // [worker][2] PromptTile: the tiles under way
  static constexpr size_t order = info + 128;                  // [kMaxOrderedTiles] tile ids, 16 bits each
  static constexpr size_t end = order + kMaxOrderedTiles * 2;
  static_assert(kMaxOrderedTiles * 4 <= worker, "the tiles' costs lie in a ring during set-up");
  static constexpr size_t bytes = end + 1024;
  static_assert(bytes <= 232448, "shared memory");
};

struct PromptTile {
  int q0, n;       // first query (of the pack) and how many (0: nothing to do)
  int k0, keys;    // the prompt's first key, keys that the last query sees
  int first;       // keys that the first query sees (may be negative)
  int bad;
  int h;           // query head
};
static_assert(sizeof(PromptTile) * 4 <= 128, "room for the tiles under way");

__device__ __forceinline__ PromptTile prompt_tile(const LatentPromptParams& p, int id) {
  int a = 0, b = p.prompts - 1;  // the last prompt whose base is at most id
  while (a < b) {
    const int m = (a + b + 1) >> 1;
    if (p.q_starts[m] / kTileRows + m <= id) a = m;
    else b = m - 1;
  }
  PromptTile t;
  const int qs = p.q_starts[a], qe = p.q_starts[a + 1], ks = p.k_starts[a], ke = p.k_starts[a + 1];
  t.q0 = t.n = t.k0 = t.keys = t.first = t.bad = t.h = 0;
  const int k = id - (qs / kTileRows + a);
  if (qs < 0 || qe < qs || qe > p.Tq || ks < 0 || ke < ks || ke > p.Tk) {
    t.bad = k == 0 || a == 0;
    return t;
  }
  if (k < 0 || static_cast<long long>(k) * kTileRows >= qe - qs) return t;
  t.q0 = qs + k * kTileRows;
  t.n = min(kTileRows, qe - t.q0);
  t.k0 = ks;
  t.first = (ke - ks) - (qe - qs) + k * kTileRows + 1;
  t.keys = max(0, t.first + t.n - 1);
  return t;
}

// The last key of [a, b) of a prompt and head (kv: its first key's row) that has a number among
// its values that is not finite, or -1.  The whole warp.
template <int D>
__device__ __noinline__ int last_odd_key(const LatentPromptParams& p, const uint16_t* kv, int a, int b) {
  constexpr int kLanes = D / 8, kKeys = 32 / kLanes;  // lanes a key, keys at once
  const int lane = threadIdx.x & 31, piece = lane % kLanes;
#pragma unroll 1
  for (int k0 = b - 1; k0 >= a; k0 -= kKeys) {
    const int key = k0 - lane / kLanes;
    const uint16_t* v = kv + static_cast<size_t>(max(key, a)) * p.heads * (2 * D) + D + piece * 8;
    const unsigned odd = __ballot_sync(0xffffffffu, key >= a && odd_halves(*reinterpret_cast<const uint4*>(v)) != 0u);
    if (odd != 0u) return k0 - (__ffs(odd) - 1) / kLanes;
  }
  return -1;
}

// One row's output from its own keys: the whole warp, a key a lane for the scores, the columns
// over the lanes for the sums, relative to the maximum so far.
template <int D>
__device__ __noinline__ void attend_row(const LatentPromptParams& p, const uint16_t* q, const uint16_t* kv,
                                        const uint16_t* k_rope, int keys, uint16_t* out) {
  constexpr int NV = D / 32;
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, l = 0.f, acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
  const size_t stride = static_cast<size_t>(p.heads) * 2 * D;
#pragma unroll 1
  for (int key0 = 0; key0 < keys; key0 += 32) {
    const int key = min(key0 + lane, keys - 1), n = min(32, keys - key0);
    const uint16_t* k = kv + key * stride;
    const uint16_t* r = k_rope + key * p.rope_stride;
    float s = 0.f;
#pragma unroll 4
    for (int i = 0; i < D; i += 8) s = dot8(*reinterpret_cast<const uint4*>(q + i), *reinterpret_cast<const uint4*>(k + i), s);
#pragma unroll 4
    for (int i = 0; i < p.rope_dim; i += 8)
      s = dot8(*reinterpret_cast<const uint4*>(q + D + i), *reinterpret_cast<const uint4*>(r + i), s);
    s *= p.scale_log2;
    float top = m;  // (the last lanes' keys repeat the last one; of NaN scores the sum tells)
    top = fmaxf(top, s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top > m) {
      const float f = exp2f(m - top);
      l *= f;
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[j] *= f;
      m = top;
    }
    const float e = lane < n ? exp2f(s - (m == -INFINITY ? 0.f : m)) : 0.f;
    l += e;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float f = __shfl_sync(0xffffffffu, e, i);
      const uint16_t* v = kv + (key0 + i) * stride + D + lane;
#pragma unroll
      for (int j = 0; j < NV; ++j) acc[j] = fmaf(f, bf16_at(v + 32 * j), acc[j]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f ? 1.f / l : l;
#pragma unroll
  for (int j = 0; j < NV; ++j) out[lane + 32 * j] = static_cast<uint16_t>(pack_bf16x2(l == 0.f ? 0.f : acc[j] * inv, 0.f));
}

// A worker's item (tile, head) in its turn `k`: they are taken in the tiles' order, every other
// round backwards.  False: there is none left; n == 0: nothing to do.
__device__ __forceinline__ bool worker_item(const LatentPromptParams& p, const uint16_t* order, int tiles, int wid, int workers,
                                            long long k, PromptTile& x) {
  const long long items = static_cast<long long>(tiles) * p.heads;
  if (k * workers >= items) return false;
  const long long i = k * workers + (k & 1 ? workers - 1 - wid : wid);
  x.n = 0;
  if (i >= items) return true;
  const int at = static_cast<int>(i / p.heads);
  x = prompt_tile(p, order != nullptr ? order[at] : p.tiles - 1 - at);
  x.h = static_cast<int>(i % p.heads);
  return true;
}

// The rows of a softmax warp (rows row0 .. + 31 of its worker's tiles, all stored) whose output is not
// finite, again, where a value behind what they see is not: at the end, when nothing waits for them.
template <int D>
__device__ __noinline__ void repair_rows(const LatentPromptParams& p, const uint16_t* order, int tiles, int wid, int workers,
                                         int row0) {
  const int lane = threadIdx.x & 31;
  PromptTile x;
#pragma unroll 1
  for (long long k = 0; worker_item(p, order, tiles, wid, workers, k, x); ++k) {
    if (row0 >= x.n) continue;
    uint16_t* out = p.out + (static_cast<size_t>(x.q0 + row0) * p.heads + x.h) * D;
    uint32_t odd = 0u;
    if (row0 + lane < x.n) {
#pragma unroll 1
      for (int i = 0; i < D; i += 8) odd |= odd_halves(*reinterpret_cast<const uint4*>(out + static_cast<size_t>(lane) * p.heads * D + i));
    }
    unsigned todo = __ballot_sync(0xffffffffu, odd != 0u);
    if (todo == 0u) continue;
    const uint16_t* kv = p.kv + (static_cast<size_t>(x.k0) * p.heads + x.h) * (2 * D);
    const int bad_key = last_odd_key<D>(p, kv, max(0, x.first + row0), x.keys);
    while (todo != 0u) {
      const int rr = __ffs(todo) - 1, sees = x.first + row0 + rr;
      todo &= todo - 1;
      if (sees > bad_key) break;  // (it sees them all: what is not finite is its own; so do those after it)
      __syncwarp();
      attend_row<D>(p, p.q + (static_cast<size_t>(x.q0 + row0 + rr) * p.heads + x.h) * (D + p.rope_dim), kv,
                    p.k_rope + static_cast<long long>(x.k0) * p.rope_stride, sees, out + static_cast<size_t>(rr) * p.heads * D);
    }
  }
}

__device__ __forceinline__ void drain(uint32_t bar, int parity) {
  const uint64_t t_0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t_0 < kWaitLimitNs) {
  }
}

template <int D>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap,
                  const __grid_constant__ CUtensorMap rmap, const __grid_constant__ LatentPromptParams p) {
  using L = PromptSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = __reduce_max_sync(0xffffffffu, tid >> 5), lane = tid & 31;
  const uint32_t rank = cluster_cta_rank();
  // producers 0 and 2, issuers or relays 1 and 3, softmax 4-7 and 8-11
  const int g = warp < 4 ? warp >> 1 : (warp - 4) >> 2;
  const uint32_t kfull = smem_addr(smem + L::bars) + g * (L::kNumBars * 8);
  const uint32_t kempty = kfull + 8 * kStages;
  const uint32_t qfull = kempty + 8 * kStages;  // [2] a tile's queries and its PromptTile are there
  const uint32_t iempty = qfull + 16;           // [2] its PromptTile was read
  const uint32_t qempty = iempty + 16;          // its last Q.K^T finished
  const uint32_t vfull = qempty + 8, vempty = vfull + 8;
  const uint32_t sfull = vempty + 8;            // Q.K^T finished (and the P.V before it)
  const uint32_t pfull = sfull + 8;             // [2] half of P written (rank 0 only)
  const uint32_t pvdone = pfull + 16;           // P.V finished
  const uint32_t efree = pvdone + 8;            // the tile's outputs have left the values' place
  const uint32_t smem_w = smem_addr(smem) + g * static_cast<uint32_t>(L::worker);
  int* misc = reinterpret_cast<int*>(smem + L::misc);
  volatile int* abort_flag = misc;
  volatile int* repair = misc + 3;  // [worker] a row's output is not finite, its sum is
  volatile PromptTile* info = reinterpret_cast<volatile PromptTile*>(smem + L::info) + 2 * g;
  uint16_t* order = reinterpret_cast<uint16_t*>(smem + L::order);
  const int workers = static_cast<int>(gridDim.x >> 1) * kWorkers;
  const int wid = static_cast<int>(blockIdx.x >> 1) + g * static_cast<int>(gridDim.x >> 1);

  if (lane == 0 && (warp == 0 || warp == 2)) {
    // rank 0's full barriers also count the relay's arrival for rank 1's copy
    const uint32_t copies = rank == 0 ? 2 : 1;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(kfull + 8 * i, copies);
      mbar_init(kempty + 8 * i, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(qfull + 8 * b, copies);
      mbar_init(iempty + 8 * b, 5);  // the softmax warps, the issuer or relay
    }
    mbar_init(qempty, 1);
    mbar_init(vfull, copies);
    mbar_init(vempty, 1);
    mbar_init(sfull, 1);
    for (int i = 0; i < 2; ++i) mbar_init(pfull + 8 * i, 8);  // four softmax warps in each CTA
    mbar_init(pvdone, 1);
    mbar_init(efree, 4);
    fence_mbarrier_init();
  }
  if (tid == 0) {
    *abort_flag = 0;
    repair[0] = repair[1] = 0;
    misc[2] = p.tiles;
  }
  if (warp == 1) tmem2_alloc(smem_addr(misc + 1), L::kTmemCols);
  // ---- tiles with the most keys first ----
  const bool ordered = p.tiles <= kMaxOrderedTiles;
  if (ordered) {
    int* cost = reinterpret_cast<int*>(smem);
    for (int i = tid; i < p.tiles; i += kThreads) {
      const PromptTile x = prompt_tile(p, i);
      cost[i] = x.n > 0 ? x.keys + 1 : 0;
      if (x.bad && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_SEGMENT);
    }
    __syncthreads();
    for (int i = tid; i < p.tiles; i += kThreads) {
      const int ci = cost[i];
      int rk = 0;
      for (int k = 0; k < p.tiles; ++k) {
        const int ck = cost[k];
        rk += (ck > ci) || (ck == ci && k > i);
      }
      order[rk] = static_cast<uint16_t>(i);
      if (ci == 0) atomicMin(misc + 2, rk);  // (from here on: nothing to do)
    }
    fence_proxy_async_smem();  // (copies will write where the costs were)
  }
  // barriers initialised and tensor memory allocated in both CTAs before any
  // thread of either uses them
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(misc[1]));

  if (warp == 0 || warp == 2) {
    // ============================== producer ==============================
    // (the launch's registers, 384 x 168, hold 128 x 80 and 256 x 208)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (lane == 0) {
      int it = 0, nk = 0, nv = 0;  // tiles; copies issued
      bool ok = true;
      PromptTile x;
      x.bad = 0;
      for (long long k = 0; ok && worker_item(p, ordered ? order : nullptr, misc[2], wid, workers, k, x); ++k) {
        if (!ordered && x.bad && x.h == 0 && rank == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_SEGMENT);
        if (x.n <= 0) continue;
        const int b = it & 1;
        if (it >= 1) ok = mbar_wait(qempty, (it - 1) & 1, abort_flag);
        if (ok && it >= 2) ok = mbar_wait(iempty + 8 * b, ((it >> 1) - 1) & 1, abort_flag);
        if (!ok) break;
        info[b].q0 = x.q0;
        info[b].n = x.n;
        info[b].k0 = x.k0;
        info[b].keys = x.keys;
        info[b].first = x.first;
        info[b].h = x.h;
        mbar_arrive_expect_tx(qfull + 8 * b, L::kQ);
        for (int c = 0; c < L::kBoxesK; ++c)
          tma_load_3d(smem_w + static_cast<uint32_t>(L::q) + c * L::kQBox, &qmap, c * kBoxCols, x.h,
                      x.q0 + static_cast<int>(rank) * kRows, qfull + 8 * b);
        ++it;
        const int nsteps = (x.keys + kStepKeys - 1) / kStepKeys;
        // keys a step ahead of the values, in the order in which the products free them
        for (int j = 0; j <= nsteps; ++j) {
          if (j < nsteps) {
            const int s = nk % kStages;
            if (nk >= kStages) ok = mbar_wait(kempty + 8 * s, ((nk / kStages) - 1) & 1, abort_flag);
            if (!ok) break;
            // this CTA's 64 keys of the step
            const uint32_t dst = smem_w + static_cast<uint32_t>(L::k) + s * L::kKStage;
            const int y = x.k0 + j * kStepKeys + static_cast<int>(rank) * 64;
            mbar_arrive_expect_tx(kfull + 8 * s, L::kKStage);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * kBoxBytes, &kvmap, c * kBoxCols, x.h, y, kfull + 8 * s);
            tma_load_2d(dst + (D / 64) * kBoxBytes, &rmap, 0, y, kfull + 8 * s);
            ++nk;
          }
          // the tile before's outputs leave through the values' place.  (Waited for once a tile, of no
          // keys too: with a phase left out, the wait for the next would take an older one for it.  it
          // counts this tile.)
          if (j == (nsteps > 0 ? 1 : 0) && it >= 2) ok = mbar_wait(efree, (it - 2) & 1, abort_flag);
          if (!ok) break;
          if (j > 0) {
            if (nv >= 1) ok = mbar_wait(vempty, (nv - 1) & 1, abort_flag);
            if (!ok) break;
            // this CTA's value columns of the step's 128 keys
            const uint32_t dst = smem_w + static_cast<uint32_t>(L::v);
            const int xv = D + static_cast<int>(rank) * kBoxCols, y = x.k0 + (j - 1) * kStepKeys;
            mbar_arrive_expect_tx(vfull, L::kVStage);
            tma_load_3d(dst, &kvmap, xv, x.h, y, vfull);
            tma_load_3d(dst + kBoxBytes, &kvmap, xv, x.h, y + 64, vfull);
            ++nv;
          }
        }
      }
      const int tiles = it;
      if (ok) {  // no more tiles
        const int b = it & 1;
        if (it >= 2) ok = mbar_wait(iempty + 8 * b, ((it >> 1) - 1) & 1, abort_flag);
        if (ok) {
          info[b].n = -1;
          mbar_arrive(qfull + 8 * b);
        }
      }
      // do not leave while a copy may still land in this CTA's memory
      if (tiles > 0) drain(qfull + 8 * ((tiles - 1) & 1), ((tiles - 1) >> 1) & 1);
      for (int k = max(0, nk - kStages); k < nk; ++k) drain(kfull + 8 * (k % kStages), (k / kStages) & 1);
      if (nv > 0) drain(vfull, (nv - 1) & 1);
    }
  } else if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (rank != 0) {
      // ========= relay of queries, keys and values (rank 1 to rank 0) ========
      if (lane == 0) {
        const uint32_t kfull0 = mapa_shared(kfull, 0), qfull0 = mapa_shared(qfull, 0), vfull0 = mapa_shared(vfull, 0);
        bool ok = true;
        for (int it = 0, nk = 0, nv = 0; ok; ++it) {
          const int b = it & 1;
          if (!mbar_wait(qfull + 8 * b, (it >> 1) & 1, abort_flag)) break;
          const int n = info[b].n, nsteps = (info[b].keys + kStepKeys - 1) / kStepKeys;
          mbar_arrive(iempty + 8 * b);
          mbar_arrive_remote(qfull0 + 8 * b);
          if (n < 0) break;
          for (int j = 0; j <= nsteps; ++j) {
            if (j < nsteps) {
              ok = mbar_wait(kfull + 8 * (nk % kStages), (nk / kStages) & 1, abort_flag);
              if (!ok) break;
              mbar_arrive_remote(kfull0 + 8 * (nk % kStages));
              ++nk;
            }
            if (j > 0) {
              ok = mbar_wait(vfull, nv & 1, abort_flag);
              if (!ok) break;
              mbar_arrive_remote(vfull0);
              ++nv;
            }
          }
        }
      }
    } else {
      // ============================ issuer (rank 0) =========================
      // (The whole warp, on values that reductions make the same in all its threads: from one
      // thread's branch, between the softmax warps, a product took 110 clocks to issue.)
      constexpr uint32_t kIdS = umma_idesc_bf16(kTileRows, kStepKeys, 0, 0);
      constexpr uint32_t kIdPV = umma_idesc_bf16(kTileRows, 128, 0, 1);
      const uint64_t qdesc = umma_desc_sw128(smem_w + static_cast<uint32_t>(L::q), 0, 1024);
      const uint64_t kdesc = umma_desc_sw128(smem_w + static_cast<uint32_t>(L::k), 0, 1024);
      const uint64_t vdesc = umma_desc_sw128(smem_w + static_cast<uint32_t>(L::v), 0, 1024);
      const uint32_t k_lo = static_cast<uint32_t>(kdesc), k_hi = static_cast<uint32_t>(kdesc >> 32);
      const uint32_t q_lo = static_cast<uint32_t>(qdesc), q_hi = static_cast<uint32_t>(qdesc >> 32);
      const uint32_t v_lo = static_cast<uint32_t>(vdesc), v_hi = static_cast<uint32_t>(vdesc >> 32);
      const uint32_t sc = tmem + L::kColS + g * 128u, oc = tmem + L::kColO + g * 128u;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag)) != 0;
      };
      auto wait2 = [&](uint32_t b1, uint32_t p1, uint32_t b2, uint32_t p2) {  // (the second as ptx.cuh asks for)
        return __all_sync(0xffffffffu, mbar_wait(b1, p1, abort_flag) && mbar_wait_cluster(b2, p2, abort_flag)) != 0;
      };
      bool ok = true;
      for (int it = 0, js = 0; ok; ++it) {
        const int qb = it & 1;
        if (!wait(qfull + 8 * qb, (it >> 1) & 1)) break;
        const int n = __reduce_max_sync(0xffffffffu, info[qb].n);
        const int nsteps = __reduce_max_sync(0xffffffffu, (info[qb].keys + kStepKeys - 1) / kStepKeys);
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty + 8 * qb);
        if (n < 0) break;
#pragma unroll 1
        for (int j = 0; j < nsteps; ++j, ++js) {
          const int s = js % kStages;
          // S, over the P that the P.V before reads
          ok = js < 1 ? wait(kfull + 8 * s, (js / kStages) & 1) : wait2(kfull + 8 * s, (js / kStages) & 1, pvdone, (js - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t kd = k_lo + ((s * L::kKStage) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16 + 2; ++kk)
            umma2_ss_warp(sc, q_lo + (((kk >> 2) * L::kQBox + (kk & 3) * 32) >> 4), q_hi,
                          kd + (((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4), k_hi, kIdS, kk > 0 ? 1u : 0u);
          if (p.rope_dim == 64) {
#pragma unroll
            for (int kk = D / 16 + 2; kk < D / 16 + 4; ++kk)
              umma2_ss_warp(sc, q_lo + (((kk >> 2) * L::kQBox + (kk & 3) * 32) >> 4), q_hi,
                            kd + (((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4), k_hi, kIdS, 1u);
          }
          umma2_commit_both_warp(sfull);
          umma2_commit_both_warp(kempty + 8 * s);
          if (j + 1 == nsteps) umma2_commit_both_warp(qempty);
          // (that all rows' P is there says too that the tile before's O has been read)
          ok = wait2(vfull, js & 1, pfull, js & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kStepKeys / 32; ++kk)
            umma2_ts_warp(oc, sc + kk * 8, v_lo + ((kk * 16 * 128) >> 4), v_hi, kIdPV, kk > 0 || j > 0 ? 1u : 0u);
          ok = wait(pfull + 8, js & 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = kStepKeys / 32; kk < kStepKeys / 16; ++kk)
            umma2_ts_warp(oc, sc + kk * 8, v_lo + ((kk * 16 * 128) >> 4), v_hi, kIdPV, 1u);
          umma2_commit_both_warp(pvdone);
          umma2_commit_both_warp(vempty);
        }
        if (nsteps == 0) umma2_commit_both_warp(qempty);
      }
      __syncwarp();
    }
  } else {
    // ============================== softmax ===============================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // thread r of a worker's four warps owns query row r of this CTA
    const int qt = warp & 3;
    const int rl = qt * 32 + lane;
    const int row = static_cast<int>(rank) * kRows + rl;
    const uint32_t lanes = static_cast<uint32_t>(qt * 32) << 16;
    const uint32_t pfull0 = mapa_shared(pfull, 0);
    const uint32_t sc = tmem + lanes + L::kColS + g * 128u, oc = tmem + lanes + L::kColO + g * 128u;
    bool ok = true;
    for (int it = 0, js = 0; ok; ++it) {
      ok = __all_sync(0xffffffffu, mbar_wait(qfull + 8 * (it & 1), (it >> 1) & 1, abort_flag));
      if (!ok) break;
      PromptTile tile;
      tile.q0 = info[it & 1].q0;
      tile.n = info[it & 1].n;
      tile.k0 = info[it & 1].k0;
      tile.keys = info[it & 1].keys;
      tile.first = info[it & 1].first;
      tile.h = info[it & 1].h;
      __syncwarp();
      if (lane == 0) mbar_arrive(iempty + 8 * (it & 1));
      if (tile.n < 0) break;
      const int nsteps = (tile.keys + kStepKeys - 1) / kStepKeys;
      const bool live = row < tile.n;
      const int hi = live ? tile.first + row : 0;  // keys that this row sees
      float m_ref = -INFINITY;  // the row's running max (log2 units), and its sum's reference
      float l = 0.f;
      for (int j = 0; j < nsteps; ++j, ++js) {
        const int kb = j * kStepKeys;
        ok = __all_sync(0xffffffffu, mbar_wait(sfull, js & 1, abort_flag));
        const bool partial = kb + kStepKeys > tile.keys;
        if (ok && partial) {
          // keys past the tile's last may hold anything: zero their value rows
          ok = __all_sync(0xffffffffu, mbar_wait(vfull, js & 1, abort_flag));
          if (ok && kb + rl >= tile.keys) {
            uint8_t* vrow = smem + g * L::worker + L::v + (rl >> 6) * kBoxBytes + (rl & 63) * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(vrow + ((c ^ rl) & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();  // (the arrival for the first half of P publishes them to the cluster)
        }
        if (!ok) break;
        tc_fence_after();
        float x[kStepKeys];
        {
          uint32_t r0[32], r1[32], r2[32], r3[32];
          tmem_ld32(sc, r0);
          tmem_ld32(sc + 32, r1);
          tmem_ld32(sc + 64, r2);
          tmem_ld32(sc + 96, r3);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            x[i] = __uint_as_float(r0[i]);
            x[32 + i] = __uint_as_float(r1[i]);
            x[64 + i] = __uint_as_float(r2[i]);
            x[96 + i] = __uint_as_float(r3[i]);
          }
        }
        const int e0 = live ? hi - kb : kStepKeys;  // visible keys of this step: below e0
        if (!__all_sync(0xffffffffu, e0 >= kStepKeys)) {
#pragma unroll
          for (int b = 0; b < kStepKeys; b += 32) {
            const uint32_t see = e0 >= b + 32 ? 0xffffffffu : e0 <= b ? 0u : (1u << (e0 - b)) - 1u;
#pragma unroll
            for (int i = 0; i < 32; ++i) x[b + i] = see >> i & 1u ? x[b + i] : -INFINITY;
          }
        }
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m8[k] = fmax3(x[k], x[8 + k], x[16 + k]);
#pragma unroll
          for (int i = 24; i < kStepKeys - 8; i += 16) m8[k] = fmax3(m8[k], x[i + k], x[i + 8 + k]);
          m8[k] = fmaxf(m8[k], x[kStepKeys - 8 + k]);
        }
        const float mraw = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
        const float mx = mraw == -INFINITY ? -INFINITY : mraw * p.scale_log2;
        float alpha = 1.f;
        if (mx != -INFINITY) {
          if (m_ref == -INFINITY) {
            m_ref = mx;
          } else if (mx > m_ref + kRescaleLog2) {
            alpha = exp2f(m_ref - mx);
            m_ref = mx;
            l *= alpha;
          }
        }
        const float nbase = m_ref == -INFINITY ? 0.f : -m_ref;
        const uint64_t c2 = f32x2(p.scale_log2, p.scale_log2), n2 = f32x2(nbase, nbase);
        if (__any_sync(0xffffffffu, alpha != 1.f) && j >= 1) {
          // rescale this row of O (the P.V of the step before ended before this step's scores came)
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t r[16];
            tmem_ld16(oc + c * 16, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
            tmem_st16(oc + c * 16, r);
          }
        }
        float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float a0v, a1v;
            f32x2_split(fma_f32x2(f32x2(x[hh * 64 + 2 * i], x[hh * 64 + 2 * i + 1]), c2, n2), a0v, a1v);
            const float e0v = ex2_approx(a0v), e1v = ex2_approx(a1v);
            s[i & 3] += e0v;
            s[(i + 2) & 3] += e1v;
            pk[i] = pack_bf16x2(e0v, e1v);
          }
          tmem_st32(sc + hh * 32, pk);
          // the products of half of P may begin
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if (hh == 0 && partial) mbar_arrive_remote_shared(pfull0);
            else mbar_arrive_remote(pfull0 + 8 * hh);
          }
        }
        l += (s[0] + s[1]) + (s[2] + s[3]);
      }
      // ---- normalise and store, half a row at a time ----
      if (ok && nsteps > 0) ok = __all_sync(0xffffffffu, mbar_wait(pvdone, (js - 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : l;  // (a NaN sum makes the row NaN)
      const bool none = l == 0.f;
      constexpr int kPieces = D / 16;  // 16-byte pieces of half a row
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t r[D / 2];
        if (nsteps > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t (&rc)[16] = *reinterpret_cast<uint32_t(*)[16]>(r + c * 16);
            tmem_ld16(oc + hf * (D / 2) + c * 16, rc);
          }
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) r[i] = 0u;
        }
        uint4 w[kPieces];
        uint32_t odd = 0u;  // bits 15 and 31: an element is not finite
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          float v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = none ? 0.f : __uint_as_float(r[8 * i + k]) * inv;
          w[i] = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                            pack_bf16x2(v[6], v[7]));
          odd |= odd_halves(w[i]);
        }
        // (a NaN sum is the row's own: all of it is NaN)
        if (live && odd != 0u && l == l) repair[g] = 1;
        // through shared memory (where the values were, whose products have ended), so that a store
        // covers whole lines
        uint8_t* mine = smem + g * L::worker + L::v + qt * (32 * 16 * kPieces);
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          *reinterpret_cast<uint4*>(mine + (lane * kPieces + (i ^ (lane & (kPieces - 1)))) * 16) = w[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int rr = (lane & ~(kPieces - 1)) + i;
          w[i] = *reinterpret_cast<const uint4*>(mine + (rr * kPieces + ((lane & (kPieces - 1)) ^ (rr & (kPieces - 1)))) * 16);
        }
        uint16_t* o = p.out + (static_cast<size_t>(tile.q0 + (row & ~(kPieces - 1))) * p.heads + tile.h) * D + hf * (D / 2) +
                      (lane & (kPieces - 1)) * 8;
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          if ((row & ~(kPieces - 1)) + i < tile.n)
            *reinterpret_cast<uint4*>(o + static_cast<size_t>(i) * p.heads * D) = w[i];
        __syncwarp();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(efree);
    }
    if (!ok) *abort_flag = 1;
    else if (__any_sync(0xffffffffu, repair[g] != 0))
      repair_rows<D>(p, ordered ? order : nullptr, misc[2], wid, workers, static_cast<int>(rank) * kRows + qt * 32);
  }
  __syncwarp();
  if (*abort_flag && lane == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
  // neither CTA frees its tensor memory or leaves while the pair's products,
  // copies or remote arrivals may still touch it
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem2_dealloc(tmem, L::kTmemCols);
}

template <int D>
cudaError_t launch_t(const CUtensorMap& qmap, const CUtensorMap& kvmap, const CUtensorMap& rmap,
                     const LatentPromptParams& p, cudaStream_t stream) {
  const int bytes = static_cast<int>(PromptSmem<D>::bytes);
  const cudaError_t err = set_max_dynamic_smem(reinterpret_cast<const void*>(prompt_kernel<D>), bytes);
  if (err != cudaSuccess) return err;
  const long long items = static_cast<long long>(p.tiles) * p.heads;
  const long long grid = 2 * std::min<long long>(items, device_sm_count() / 2);  // a cluster a pair of SMs
  if (grid <= 0) return cudaErrorInvalidValue;
  prompt_kernel<D><<<static_cast<unsigned>(grid), kThreads, bytes, stream>>>(qmap, kvmap, rmap, p);
  return cudaGetLastError();
}

}  // namespace

int latent_prompt_tile_rows() { return kTileRows; }

cudaError_t launch_latent_prompt(const CUtensorMap& qmap, const CUtensorMap& kvmap, const CUtensorMap& rmap,
                                 const LatentPromptParams& p, cudaStream_t stream) {
  return p.head_dim == 64 ? launch_t<64>(qmap, kvmap, rmap, p, stream) : launch_t<128>(qmap, kvmap, rmap, p, stream);
}

}  // namespace lnk
