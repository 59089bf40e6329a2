// Attention over a paged latent cache in tiles of 128 query rows, for tokens of more than 64
// heads and for launches of many prompt tokens (what it computes and how the pages are
// shared out: latent_attn.cu).
//
// A pair of SMs takes a tile as 2-SM products of M = 128 rows: CTA r of the pair holds rows
// 64 r .. 64 r + 63 in its tensor memory, where 128 lanes are the 64 rows twice, the second
// time for the second half of the columns.  Per page of 64 keys
//   S[128 x 64]  = Q K^T   K: CTA r holds keys 32 r .. + 31, all numbers, K-major;
//   O[128 x C]  += P V     V: CTA r holds all 64 keys, half r of the latent, MN-major;
// so a page is copied 1.9 times into the pair's shared memory, and a row's 512 values take
// 256 columns (with all rows on one SM they would fill tensor memory).  Keys and values have
// rings of their own: keys leave after Q.K^T, values after P.V a softmax later.
// (The one-SM kernel reads a page and multiplies it for 64 rows in 2550 clocks at best, on
// each of two SMs for 128 rows; these products take 1610 for the pair: operands of a 2-SM
// product are read from both shared memories at once.)
//
// Warps: 0 loads keys and query rows, 2 values (each CTA its own); 1 issues the products in
// rank 0 and tells rank 0 of rank 1's keys and queries in rank 1, where warp 3 does so for
// values; 4-7 softmax: thread L owns row L % 64 of its CTA and keys 32 (L / 64) .. + 31 of a page,
// and that row's half L / 64 of O.  Scores and probabilities have two buffers each.
// (Rank 0's products read rank 1's probabilities from rank 1's shared memory.  The softmax warps
// order their stores before the async proxy and arrive at rank 0's barrier with a release of
// shared memory alone to the cluster; a release of all memory took a barrier of 1500 to 3500
// clocks, in these warps or in a relay's: 32 rows of 128 heads 89 us, with the join, and 56 now.)
//
// Bound: the products' operands (the pipe with its reads is active 73% of a step of 272 prompt
// tokens of 64 heads and 32 decode rows, 0.12 Tflop in 125 us, the join 10 more), and the tiles'
// ends, which the one accumulator waits for.  32 rows of 128 heads, 154 MB: 45 us, of which the
// start takes 8.5 and a unit's end 2.4, and the join 10 more.
#include "latent_units.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;          // rows of a CTA
constexpr int kSoftBar = 1;

template <int NB>
struct PairSmem {
  static constexpr int kChunks = 2 * NB + 1;              // 64 numbers of a row each; the last: the rotated ones
  static constexpr int kRg = kChunks * 1024;              // eight keys
  static constexpr int kK = 4 * kRg;                      // a page's keys of this CTA
  static constexpr int kVRg = NB * 1024;                  // eight keys' values, this CTA's half
  static constexpr int kV = 8 * kVRg;
  static constexpr int kQ = kChunks * kRows * 128;
  static constexpr int kP = kRows * 128;
  static constexpr int kMisc = 2048;
  static constexpr int kBudget = 232448 - 1024 - kMisc - kQ - 2 * kP;
  static constexpr int kStages = kBudget / (kK + kV) < 4 ? kBudget / (kK + kV) : 4;
  static constexpr size_t k = 0;
  static constexpr size_t v = k + size_t(kStages) * kK;
  static constexpr size_t q = v + size_t(kStages) * kV;
  static constexpr size_t p = q + kQ;
  static constexpr size_t bars = p + 2 * kP;
  // kfull, kempty, vfull, vempty [stages], sfull[2], pfull[2], pvdone[2], qfull, qempty, fin
  static constexpr int kNumBars = 4 * kStages + 9;
  static constexpr size_t ref = bars + 8 * kNumBars;      // [64] a row's first score; in a raise the maxima
  static constexpr size_t pair = ref + 4 * kRows;         // [2][64] what a row's two threads tell each other
  static constexpr size_t misc = pair + 8 * kRows;        // abort, tensor memory, beat, share
  static constexpr size_t end = misc + 256;
  static_assert(end - bars <= kMisc, "barriers and row data");
  static_assert(kStages >= 2, "stages");
  static constexpr size_t bytes = bars + kMisc + 1024;
  static constexpr uint32_t kColS = NB * 64;              // after O
  static constexpr uint32_t kCols = NB * 64 + 64 <= 128 ? 128 : NB * 64 + 64 <= 256 ? 256 : 512;
};

__device__ __forceinline__ void drain(uint32_t bar, int parity) {
  const uint64_t t_0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t_0 < kWaitLimitNs) {
  }
}

template <int NB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    pair_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap rmap,
                const __grid_constant__ LatentParams p) {
  using L = PairSmem<NB>;
  constexpr int kStages = L::kStages;
  constexpr int C = NB * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t kfull = smem_addr(smem + L::bars);
  const uint32_t kempty = kfull + 8 * kStages, vfull = kempty + 8 * kStages, vempty = vfull + 8 * kStages;
  const uint32_t sfull = vempty + 8 * kStages;  // [2] scores of a page
  const uint32_t pfull = sfull + 16;            // [2] probabilities of a page (rank 0 only)
  const uint32_t pvdone = pfull + 16;           // [2] the value product of a page
  const uint32_t qfull = pvdone + 16, qempty = qfull + 8, fin = qempty + 8;
  float* s_ref = reinterpret_cast<float*>(smem + L::ref);
  float* s_pair = reinterpret_cast<float*>(smem + L::pair);
  int* misc = reinterpret_cast<int*>(smem + L::misc);
  volatile int* abort_flag = misc;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int tid = threadIdx.x, warp = __reduce_max_sync(0xffffffffu, tid >> 5), lane = tid & 31;
  const int rank = static_cast<int>(cluster_cta_rank());
  const int team = static_cast<int>(blockIdx.x >> 1) / p.head_blocks, hb = static_cast<int>(blockIdx.x >> 1) % p.head_blocks;

  if (tid == 0) {
    // rank 0's full barriers also count the relay's arrival for rank 1's copy
    const uint32_t copies = rank == 0 ? 2 : 1;
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(kfull + 8 * i, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(kfull + 8 * i, copies);
      mbar_init(vfull + 8 * i, copies);
    }
    mbar_init(qfull, copies);
    for (int i = 0; i < 2; ++i) mbar_init(pfull + 8 * i, 8);  // the softmax warps of both CTAs
    abort_flag[0] = abort_flag[kBeat] = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) tmem2_alloc(smem_addr(misc + 1), L::kCols);
  // positions, rows and the table are read before the wait for the kernel before this one
  const Shares shares = count_shares<kThreads>(p, team, misc + 4);
  // barriers initialised and tensor memory allocated in both CTAs before any
  // thread of either uses them
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(misc[1]));
  const Share* share = share_of(misc + 4);
  int t = share->t, j0 = share->j;
  long long left = static_cast<long long>(share->left);

  // what the kernel before this one on the stream writes is touched from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (shares.bad && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, shares.bad);
  if (tid == 0 && rank == 0 && hb == 0 && !p.whole) write_cut(p, team, t, left > 0 ? j0 : 0, shares.per);

  // Walks the share: f(unit, its pages here, unit's number) for each of its units in turn.
  auto units = [&](auto&& f) {
    for (int u = 0; left > 0; ++u) {
      const Unit un = unit_at(p, t);
      const int n = static_cast<int>(min(left, static_cast<long long>(un.np - j0)));
      if (!f(un, n, u)) break;
      left -= n;
      t += un.nt;
      j0 = 0;
    }
  };
  // The page of table entry `i` of a unit here, or page 0 for one that is not there (its keys are
  // masked and its values zeroed).
  auto page_of = [&](const Unit& un, int i, bool report) {
    int page = un.row >= 0 ? p.table[static_cast<long long>(un.row) * p.pages_per_row + un.first + j0 + i] : 0;
    if (page < 0 || page >= p.num_pages) {
      if (report && hb == 0 && rank == 0 && p.status != nullptr && page_seen(p, t, un.nt, un.first + j0 + i))
        atomicOr(p.status, LNK_DEV_BAD_PAGE);
      page = 0;
    }
    return page;
  };

  if (warp == 0) {
    // ===================== producer of keys and queries =====================
    if (lane == 0) {
      int g = 0, asked = 0;  // pages; query tiles asked for
      auto load_q = [&](int t) {
        mbar_arrive_expect_tx(qfull, L::kQ);
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_2d(smem_addr(smem + L::q) + c * (kRows * 128), &qmap, c * kBoxCols, t * p.heads + hb * 2 * kRows + rank * kRows,
                      qfull);
        ++asked;
      };
      if (left > 0) load_q(t);
      units([&](const Unit& un, int n, int u) {
        for (int i = 0; i < n; ++i, ++g) {
          const int page = page_of(un, i, true);
          const int st = g % kStages;
          if (g >= kStages && !wait_with_beat(kempty + 8 * st, ((g / kStages) - 1) & 1, abort_flag)) return false;
          const uint32_t dst = smem_addr(smem + L::k) + st * L::kK, fb = kfull + 8 * st;
          mbar_arrive_expect_tx(fb, L::kK);
          if (p.rope_dim == 64) {
            tma_load_4d(dst, &kmap, 0, 0, 0, page * 8 + rank * 4, fb);
          } else {
            for (int k = 0; k < 4; ++k) {
              tma_load_4d(dst + k * L::kRg, &kmap, 0, 0, 0, page * 8 + rank * 4 + k, fb);
              tma_load_2d(dst + k * L::kRg + 2 * NB * 1024, &rmap, C, page * kPage + (rank * 4 + k) * 8, fb);
            }
          }
          if (i == 0 && u > 0) {
            if (!wait_with_beat(qempty, (u - 1) & 1, abort_flag)) {
              ++g;  // (this page was asked for)
              return false;
            }
            load_q(t);
          }
        }
        return true;
      });
      // do not leave while a copy may still land in this CTA's memory
      for (int k = max(0, g - kStages); k < g; ++k) drain(kfull + 8 * (k % kStages), (k / kStages) & 1);
      if (asked > 0) drain(qfull, (asked - 1) & 1);
    }
  } else if (warp == 2) {
    // ========================== producer of values ==========================
    if (lane == 0) {
      int g = 0;
      units([&](const Unit& un, int n, int) {
        for (int i = 0; i < n; ++i, ++g) {
          const int page = page_of(un, i, false);
          const int st = g % kStages;
          if (g >= kStages && !wait_with_beat(vempty + 8 * st, ((g / kStages) - 1) & 1, abort_flag)) return false;
          mbar_arrive_expect_tx(vfull + 8 * st, L::kV);
          tma_load_4d(smem_addr(smem + L::v) + st * L::kV, &vmap, 0, 0, rank * NB, page * 8, vfull + 8 * st);
        }
        return true;
      });
      for (int k = max(0, g - kStages); k < g; ++k) drain(vfull + 8 * (k % kStages), (k / kStages) & 1);
    }
  } else if (warp == 3 || (warp == 1 && rank != 0)) {
    // ====================== relays of rank 1 to rank 0 ======================
    if (rank != 0 && lane == 0) {
      const uint32_t mine = warp == 1 ? kfull : vfull, theirs = mapa_shared(mine, 0);
      const uint32_t qfull0 = mapa_shared(qfull, 0);
      int g = 0;
      units([&](const Unit&, int n, int u) {
        if (warp == 1) {
          if (!wait_with_beat(qfull, u & 1, abort_flag)) return false;
          mbar_arrive_remote(qfull0);
        }
        for (int i = 0; i < n; ++i, ++g) {
          if (!wait_with_beat(mine + 8 * (g % kStages), (g / kStages) & 1, abort_flag)) return false;
          mbar_arrive_remote(theirs + 8 * (g % kStages));
        }
        return true;
      });
    }
  } else if (warp == 1) {
    // ======================= products' issuer (rank 0) ======================
    // The whole warp runs this, on values that are the same in all its threads (latent_attn.cu).
    constexpr uint32_t kIdS = umma_idesc_bf16(2 * kRows, kPage, 0, 0);
    constexpr uint32_t kIdPV = umma_idesc_bf16(2 * kRows, 256, 0, 1);
    constexpr uint32_t kIdPV1 = umma_idesc_bf16(2 * kRows, 128, 0, 1);  // (the odd 64 numbers of a half)
    const uint64_t kdesc = umma_desc_sw128(smem_addr(smem + L::k), 0, L::kRg);
    const uint64_t qdesc = umma_desc_sw128(smem_addr(smem + L::q), 0, 1024);
    const uint64_t vdesc = umma_desc_sw128(smem_addr(smem + L::v), 1024, L::kVRg);
    const uint64_t pdesc = umma_desc_sw128(smem_addr(smem + L::p), 0, 1024);
    const uint32_t k_lo = static_cast<uint32_t>(kdesc), k_hi = static_cast<uint32_t>(kdesc >> 32);
    const uint32_t q_lo = static_cast<uint32_t>(qdesc), q_hi = static_cast<uint32_t>(qdesc >> 32);
    const uint32_t v_lo = static_cast<uint32_t>(vdesc), v_hi = static_cast<uint32_t>(vdesc >> 32);
    const uint32_t p_lo = static_cast<uint32_t>(pdesc), p_hi = static_cast<uint32_t>(pdesc >> 32);
    auto uniform = [](int x) { return __reduce_max_sync(0xffffffffu, x); };
    auto done = [](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_test_wait_cluster(bar, parity)) != 0;
    };
    // scores of page s and the value product of page v <= s, in whatever order they become ready
    int s = 0, v = 0, u = 0;
    int ut = 0, un = 0, ui = 0;  // tokens and pages (of this share) of unit u, page s in it
    uint32_t first = 0u;         // bit s & 1: page s is its unit's first here
    int more = uniform(left > 0);
    if (more != 0) {
      const Unit x = unit_at(p, t);
      ut = x.nt;
      un = uniform(static_cast<int>(min(left, static_cast<long long>(x.np - j0))));
    }
    uint64_t t0 = 0;
    uint32_t idle = 0;
    while (more != 0 || v < s) {
      bool did = false;
      if (v < s && done(pfull + 8 * (v & 1), (v >> 1) & 1) && done(vfull + 8 * (v % kStages), (v / kStages) & 1)) {
        tc_fence_after();
        const uint32_t vd = v_lo + (((v % kStages) * L::kV) >> 4), pd = p_lo + (((v & 1) * L::kP) >> 4);
        const uint32_t keep = first >> (v & 1) & 1u ? 0u : 1u;
#pragma unroll 1
        for (int kk = 0; kk < kPage / 16; ++kk) {
          const uint32_t sum = kk > 0 ? 1u : keep;
#pragma unroll
          for (int b = 0; b < NB / 2; ++b)
            umma2_ss_warp(tmem + b * 128, pd + ((kk * 32) >> 4), p_hi, vd + ((kk * 2 * L::kVRg + b * 2048) >> 4), v_hi, kIdPV,
                          sum);
          if constexpr (NB % 2 == 1)
            umma2_ss_warp(tmem + (NB / 2) * 128, pd + ((kk * 32) >> 4), p_hi,
                          vd + ((kk * 2 * L::kVRg + (NB / 2) * 2048) >> 4), v_hi, kIdPV1, sum);
        }
        umma2_commit_both_warp(vempty + 8 * (v % kStages));
        umma2_commit_both_warp(pvdone + 8 * (v & 1));
        ++v;
        did = true;
      }
      // (two score buffers: page s - 2 has been read once its value product was issued)
      if (more != 0 && s <= v + 1 && done(kfull + 8 * (s % kStages), (s / kStages) & 1) && (ui > 0 || done(qfull, u & 1))) {
        tc_fence_after();
        const uint32_t sc = tmem + L::kColS + (s & 1) * 32;
        uint32_t kd = k_lo + (((s % kStages) * L::kK) >> 4), qd = q_lo;
#pragma unroll 1
        for (int c = 0; c < 2 * NB; ++c, kd += 1024 >> 4, qd += (kRows * 128) >> 4) {
          umma2_ss_warp(sc, qd, q_hi, kd, k_hi, kIdS, c > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) umma2_ss_warp(sc, qd + ((kk * 32) >> 4), q_hi, kd + ((kk * 32) >> 4), k_hi, kIdS, 1u);
        }
        umma2_ss_warp(sc, qd, q_hi, kd, k_hi, kIdS, 1u);
        umma2_ss_warp(sc, qd + (32 >> 4), q_hi, kd + (32 >> 4), k_hi, kIdS, 1u);
        if (p.rope_dim == 64) {
          umma2_ss_warp(sc, qd + (64 >> 4), q_hi, kd + (64 >> 4), k_hi, kIdS, 1u);
          umma2_ss_warp(sc, qd + (96 >> 4), q_hi, kd + (96 >> 4), k_hi, kIdS, 1u);
        }
        umma2_commit_both_warp(sfull + 8 * (s & 1));
        umma2_commit_both_warp(kempty + 8 * (s % kStages));
        first = (first & ~(1u << (s & 1))) | (ui == 0 ? 1u << (s & 1) : 0u);
        ++s;
        if (++ui == un) {  // the unit's last scores: its query rows may go
          umma2_commit_both_warp(qempty);
          left -= un;
          t += ut;
          ui = 0;
          ++u;
          more = uniform(left > 0);
          if (more != 0) {
            const Unit x = unit_at(p, t);
            ut = x.nt;
            un = uniform(static_cast<int>(min(left, static_cast<long long>(x.np))));
          }
        }
        did = true;
      }
      if (did) {
        idle = 0;
      } else if ((++idle & 255u) == 0) {
        if (idle == 256u) t0 = global_timer_ns();
        const bool late = global_timer_ns() - t0 > kWaitLimitNs || idle >= kWaitLimitIters;
        if (__any_sync(0xffffffffu, (late && !beat_is_recent(abort_flag + kBeat)) || *abort_flag != 0)) {
          *abort_flag = 1;
          break;
        }
      }
    }
    // no product is in flight when the tensor memory goes
    umma2_commit_both_warp(fin);
    wait_with_beat(fin, 0, abort_flag);
    __syncwarp();
  } else {
    // ============================== softmax ===============================
    const int qt = warp & 3;
    const int row = (qt & 1) * 32 + lane, half = qt >> 1;
    const int rr = rank * kRows + row;               // row of the tile
    const uint32_t lanes = static_cast<uint32_t>(qt * 32) << 16;
    const uint32_t pfull0 = mapa_shared(pfull, 0);
    const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
    uint8_t* prow = smem + L::p + row * 128;
    bool ok = true;
    int g = 0;
    units([&](const Unit& un, int n, int) {
      const int nrows = min(2 * kRows, un.nt * p.heads - hb * 2 * kRows);
      const int rowbase = t * p.heads + hb * 2 * kRows;
      const bool direct = j0 == 0 && n == un.np;
      // keys that this row sees (rows past the unit's: everything, nobody reads them)
      int lo = 0, hi = 0x7fffffff;
      if (rr < nrows) {
        int r0;
        token_keys(p, t + (hb * 2 * kRows + rr) / p.heads, r0, lo, hi);
      }
      const int32_t* trow = p.table + static_cast<long long>(max(un.row, 0)) * p.pages_per_row;
      // minus the reference (0 while there is none; rows past the unit's have no weights, and nothing to
      // raise), this thread's part of the sum
      float nref = rr < nrows ? 0.f : -INFINITY, l = 0.f;
      bool unset = rr < nrows && hi > lo;  // no reference yet, and keys to see
      bool force = true;                   // some row of the CTA has none
      if (half == 0) s_ref[row] = -INFINITY;
      named_barrier_sync(kSoftBar, 128);
      for (int i = 0; i < n; ++i, ++g) {
        const int lp = un.first + j0 + i, kb = lp * kPage, k0 = kb + half * 32;
        const int page = un.row >= 0 ? trow[lp] : -1;
        const bool held = page >= 0 && page < p.num_pages;
        ok = __all_sync(0xffffffffu, wait_with_beat(sfull + 8 * (g & 1), (g >> 1) & 1, abort_flag));
        tc_fence_after();
        uint32_t r[32];
        if (ok) {
          tmem_ld32(tmem + lanes + L::kColS + (g & 1) * 32, r);
          tmem_ld_wait();
        }
        if (!(held && kb >= un.in_lo && kb + kPage <= un.in_hi)) {
          const int a = held ? lo - k0 : 32, e = hi - k0;
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x < a || x >= e) r[x] = 0xFF800000u;
        }
        if (force) {
          const int f = max(lo, kb) - k0;  // the row's first key of this page
          if (f >= 0 && f < 32) {
            float x0 = __uint_as_float(r[0]);
            if (f > 0) {
#pragma unroll
              for (int x = 1; x < 32; ++x)
                if (x == f) x0 = __uint_as_float(r[x]);
            }
            s_ref[row] = x0;
          }
          named_barrier_sync(kSoftBar, 128);
          const float f0 = s_ref[row];
          if (unset && f0 > -INFINITY) {  // (a NaN score: the maximum of the others, below)
            nref = fmaf(-f0, p.scale_log2, -kAheadLog2);
            unset = false;
          }
        }
        float a[32];
        float mx = -INFINITY;
        auto exponents = [&]() {
          const uint64_t n2 = f32x2(nref, nref);
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(r[x]), __uint_as_float(r[x + 1])), scale2, n2), a[x], a[x + 1]);
            mx = fmax3(mx, a[x], a[x + 1]);
          }
        };
        exponents();
        // (a row without a reference that sees a score all the same: its first one is -inf or NaN)
        const bool raise = unset ? mx > -INFINITY : mx > kRaiseLog2;
        if (named_barrier_or(kSoftBar, 128, raise || !ok)) {
          // ---- references raised (or set) with the page's maximum ----
          if (g > 0 && ok) ok = __all_sync(0xffffffffu, wait_with_beat(pvdone + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, abort_flag));
          if (named_barrier_or(kSoftBar, 128, !ok)) {
            ok = false;
            return false;
          }
          tc_fence_after();
          float m = -INFINITY;
#pragma unroll
          for (int x = 0; x < 32; ++x) m = fmaxf(m, __uint_as_float(r[x]));
          s_pair[half * kRows + row] = m;
          named_barrier_sync(kSoftBar, 128);
          m = fmaxf(m, s_pair[(half ^ 1) * kRows + row]);
          float f = 1.f;
          if (m != -INFINITY) {
            m *= p.scale_log2;
            if (unset) {
              nref = -m - kAheadLog2;
              unset = false;
            } else if (m + nref > kRaiseLog2) {
              f = ex2_approx((-m - kAheadLog2) - nref);
              l *= f;
              nref = -m - kAheadLog2;
            }
          }
          if (__any_sync(0xffffffffu, f != 1.f) && i > 0) {
#pragma unroll 1
            for (int c = 0; c < NB * 64; c += 16) {
              uint32_t v[16];
              tmem_ld16(tmem + lanes + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
              tmem_st16(tmem + lanes + c, v);
            }
            tmem_st_wait();
          }
          exponents();
        }
        if (force) force = named_barrier_or(kSoftBar, 128, unset);
        // ---- P into shared memory, once the product of two pages before has read what is there ----
        if (g > 1) ok = __all_sync(0xffffffffu, wait_with_beat(pvdone + 8 * (g & 1), ((g - 2) >> 1) & 1, abort_flag));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float e0 = ex2_approx(a[8 * c + 2 * k]), e1 = ex2_approx(a[8 * c + 2 * k + 1]);
            l += e0 + e1;
            w[k] = pack_bf16x2(e0, e1);
          }
          *reinterpret_cast<uint4*>(prow + (g & 1) * L::kP + (((half * 4 + c) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        // ---- value rows that no token of the unit sees may hold anything: zero ----
        if (!(held && kb >= un.kmin && kb + kPage <= un.kmax)) {
          ok = ok && __all_sync(0xffffffffu, wait_with_beat(vfull + 8 * (g % kStages), (g / kStages) & 1, abort_flag));
          uint8_t* v = smem + L::v + (g % kStages) * L::kV;
          // rows [0, below) and [above, 64), 16 bytes of a row a thread (eight threads a line)
          const int below = held ? min(kPage, max(0, un.kmin - kb)) : kPage;
          const int above = held ? max(below, min(kPage, un.kmax - kb)) : kPage;
          const int out = ok ? below + kPage - above : 0, sid = tid - 128;
#pragma unroll 1
          for (int k = sid >> 3; k < out; k += 16) {
            const int key = k < below ? k : k - below + above;
            uint8_t* to = v + (key >> 3) * L::kVRg + (key & 7) * 128 + (sid & 7) * 16;
#pragma unroll
            for (int c = 0; c < NB; ++c) *reinterpret_cast<uint4*>(to + c * 1024) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_shared(pfull0 + 8 * (g & 1));
      }
      // ---- the unit's end: sums joined, outputs or partial sums stored ----
      if (ok) ok = __all_sync(0xffffffffu, wait_with_beat(pvdone + 8 * ((g - 1) & 1), ((g - 1) >> 1) & 1, abort_flag));
      if (named_barrier_or(kSoftBar, 128, !ok)) {
        ok = false;
        return false;
      }
      tc_fence_after();
      s_pair[half * kRows + row] = l;
      named_barrier_sync(kSoftBar, 128);
      const float sum = s_pair[row] + s_pair[kRows + row];
      const float inv = sum > 0.f ? 1.f / sum : sum;  // (a NaN sum makes the row NaN)
      const size_t slot = direct ? 0 : (static_cast<size_t>(2 * team + (j0 == 0 ? 1 : 0)) * p.head_blocks + hb) * p.slot_rows;
      if (!direct && half == 0) {
        p.ml[(slot + rr) * 2] = sum == 0.f ? -INFINITY : -nref;
        p.ml[(slot + rr) * 2 + 1] = sum;
      }
      if (half == 0) s_ref[row] = inv;
      named_barrier_sync(kSoftBar, 128);
      // 16 rows and 64 numbers a step: a thread gets numbers 8 i + 2 (lane % 4), + 1 of rows lane / 4
      // and lane / 4 + 8.  (A loop of few instructions: they are cold when a unit ends.)
      unsigned odd[4];  // of rows 8 k .. + 7 of the warp's, four bits each: not all is finite
      const int wrow = (qt & 1) * 32 + (lane >> 2), ca = 2 * (lane & 3);
#pragma unroll 1
      for (int h16 = 0; h16 < 2; ++h16) {
        float bad0 = 0.f, bad1 = 0.f;  // 0 times every number: NaN once one is not finite
        const int ra = wrow + h16 * 16, rb = ra + 8;
        const bool see_a = rank * kRows + ra < nrows, see_b = rank * kRows + rb < nrows;
        const float fa = direct ? s_ref[ra] : 1.f, fb = direct ? s_ref[rb] : 1.f;
#pragma unroll 1
        for (int c = 0; c < NB; ++c) {
          uint32_t v[32];
          tmem_ld_16x256b(tmem + lanes + (static_cast<uint32_t>(h16 * 16) << 16) + c * 64, v);
          tmem_ld_wait();
          const int d = half * (C / 2) + c * 64;
          if (direct) {
            uint32_t wa[8], wb[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float a0 = __uint_as_float(v[4 * i]) * fa, a1 = __uint_as_float(v[4 * i + 1]) * fa;
              const float b0 = __uint_as_float(v[4 * i + 2]) * fb, b1 = __uint_as_float(v[4 * i + 3]) * fb;
              bad0 = fmaf(a0, 0.f, fmaf(a1, 0.f, bad0));
              bad1 = fmaf(b0, 0.f, fmaf(b1, 0.f, bad1));
              wa[i] = fa == 0.f ? 0u : pack_bf16x2(a0, a1);
              wb[i] = fb == 0.f ? 0u : pack_bf16x2(b0, b1);
            }
            // four lanes trade: lane l gets eight numbers of groups l and 4 + l
#pragma unroll
            for (int b = 1; b < 4; b <<= 1) {
              const bool up = (lane & b) != 0;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                if (k & b) continue;
                const uint32_t ga = __shfl_xor_sync(0xffffffffu, up ? wa[k] : wa[k | b], b);
                const uint32_t gb = __shfl_xor_sync(0xffffffffu, up ? wb[k] : wb[k | b], b);
                if (up) {
                  wa[k] = ga;
                  wb[k] = gb;
                } else {
                  wa[k | b] = ga;
                  wb[k | b] = gb;
                }
              }
            }
            uint16_t* o = p.out + static_cast<size_t>(rowbase + rank * kRows + ra) * C + d + (lane & 3) * 8;
            if (see_a) {
              *reinterpret_cast<uint4*>(o) = make_uint4(wa[0], wa[1], wa[2], wa[3]);
              *reinterpret_cast<uint4*>(o + 32) = make_uint4(wa[4], wa[5], wa[6], wa[7]);
            }
            if (see_b) {
              *reinterpret_cast<uint4*>(o + 8 * C) = make_uint4(wb[0], wb[1], wb[2], wb[3]);
              *reinterpret_cast<uint4*>(o + 8 * C + 32) = make_uint4(wb[4], wb[5], wb[6], wb[7]);
            }
          } else {
            // two lanes trade: the even one gets four numbers of group 2 i, the odd one of 2 i + 1
            const bool up = (lane & 1) != 0;
            float* o = p.o + (slot + rank * kRows + ra) * C + d + (up ? ca + 6 : ca);
            auto trade = [&](uint32_t x0, uint32_t x1, uint32_t y0, uint32_t y1) {
              const uint32_t g0 = __shfl_xor_sync(0xffffffffu, up ? x0 : y0, 1), g1 = __shfl_xor_sync(0xffffffffu, up ? x1 : y1, 1);
              return up ? make_uint4(g0, g1, y0, y1) : make_uint4(x0, x1, g0, g1);
            };
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t* x = v + 8 * i;  // groups 2 i and 2 i + 1
              const uint4 wa = trade(x[0], x[1], x[4], x[5]), wb = trade(x[2], x[3], x[6], x[7]);
#pragma unroll
              for (int k = 0; k < 8; k += 4) {
                bad0 = fmaf(__uint_as_float(x[k]), 0.f, fmaf(__uint_as_float(x[k + 1]), 0.f, bad0));
                bad1 = fmaf(__uint_as_float(x[k + 2]), 0.f, fmaf(__uint_as_float(x[k + 3]), 0.f, bad1));
              }
              if (see_a) *reinterpret_cast<uint4*>(o + 16 * i) = wa;
              if (see_b) *reinterpret_cast<uint4*>(o + 8 * C + 16 * i) = wb;
            }
          }
        }
        const unsigned ba = __ballot_sync(0xffffffffu, see_a && bad0 != bad0), bb = __ballot_sync(0xffffffffu, see_b && bad1 != bad1);
        if (h16 == 0) {
          odd[0] = ba;
          odd[1] = bb;
        } else {
          odd[2] = ba;
          odd[3] = bb;
        }
      }
      if ((odd[0] | odd[1] | odd[2] | odd[3]) != 0u) {
        const int seg_lo = max(un.kmin, (un.first + j0) * kPage), seg_hi = min(un.kmax, (un.first + j0 + n) * kPage);
        const int2 bad_keys = odd_keys<true>(p, trow, seg_lo, seg_hi, __reduce_max_sync(0xffffffffu, hi > lo ? lo : 0),
                                       __reduce_min_sync(0xffffffffu, hi > lo ? hi : 0x7fffffff), abort_flag);
#pragma unroll 1
        for (int k = 0; k < 32; ++k) {
          const unsigned m = k < 16 ? (k < 8 ? odd[0] : odd[1]) : (k < 24 ? odd[2] : odd[3]);
          const float total = __shfl_sync(0xffffffffu, sum, k);
          if ((m >> (4 * (k & 7)) & 15u) == 0u || total != total) continue;  // (a NaN sum is the row's own)
          const int lo_k = __shfl_sync(0xffffffffu, lo, k), hi_k = __shfl_sync(0xffffffffu, hi, k);
          // (so is what is not finite of a row that sees all such keys; one that sees nothing gets its zeros)
          if (hi_k > lo_k && lo_k <= bad_keys.x && hi_k > bad_keys.y) continue;
          const int ro = rank * kRows + (qt & 1) * 32 + k, w = p.latent_dim + p.rope_dim;
          __syncwarp();
          float acc[2 * NB];
          attend_again<2 * NB, 32, true>(p, p.q + static_cast<size_t>(rowbase + ro) * w, trow, max(lo_k, seg_lo), min(hi_k, seg_hi),
                                   __shfl_sync(0xffffffffu, nref, k), half * (C / 2) + lane, acc, abort_flag);
          const float f = __shfl_sync(0xffffffffu, inv, k);
#pragma unroll
          for (int i = 0; i < 2 * NB; ++i) {
            const int d = half * (C / 2) + lane + 32 * i;
            if (direct) p.out[static_cast<size_t>(rowbase + ro) * C + d] = static_cast<uint16_t>(pack_bf16x2(acc[i] * f, 0.f));
            else p.o[(slot + ro) * C + d] = acc[i];
          }
        }
      }
      tc_fence_before();
      named_barrier_sync(kSoftBar, 128);  // (the rows' data may be written again)
      return true;
    });
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  if (*abort_flag && lane == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
  // neither CTA frees its tensor memory or leaves while the pair's products,
  // copies or remote arrivals may still touch it
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem2_dealloc(tmem, L::kCols);
}

template <int NB>
cudaError_t launch_t(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap, const CUtensorMap& rmap,
                     const LatentParams& p, cudaStream_t stream) {
  const int bytes = static_cast<int>(PairSmem<NB>::bytes);
  cudaError_t err = set_max_dynamic_smem(reinterpret_cast<const void*>(pair_kernel<NB>), bytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * p.teams * p.head_blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, pair_kernel<NB>, qmap, kmap, vmap, rmap, p);
  if (err != cudaSuccess) return err;
  return launch_latent_join(p, stream);
}

}  // namespace

cudaError_t launch_latent_pair(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const CUtensorMap& rmap, const LatentParams& p, cudaStream_t stream) {
  switch (p.latent_dim / 128) {
    case 1: return launch_t<1>(qmap, kmap, vmap, rmap, p, stream);
    case 2: return launch_t<2>(qmap, kmap, vmap, rmap, p, stream);
    case 3: return launch_t<3>(qmap, kmap, vmap, rmap, p, stream);
    case 4: return launch_t<4>(qmap, kmap, vmap, rmap, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
