// Attention over a paged latent cache, absorbed form: every query head scores the
// whole row [c, k] of a token and sums the c,
//     s_hj = scale q_h . [c_j, k_j],   o_h = sum_j softmax(s_h)_j c_j.
// All heads (and all tokens of a prompt piece) share the keys, so a tile takes up to
// N = 64 query rows of consecutive (token, head) pairs that see one table row, and
// streams the row's pages (64 keys) once for all of them.
//
// The products are turned over, so that the accumulators' size follows the number of
// query rows (C = 512 values of 64 rows are half of the tensor memory; with the rows
// on the tensor-memory lanes 128 rows would fill all of it and leave no scores):
//   S^T[64 keys x N]  = K Q^T    K: the page, K-major; Q: the rows, K-major;
//   O^T[C x N]       += V^T P^T  V: the same page, read MN-major, 128 numbers of c a
//                                product; P^T: bf16, one row of N a key.
// A page therefore lies in shared memory once, as keys and as values: [8 keys][64 numbers]
// of 1 KB each, so that what a copy of 16 keys reads is contiguous in the pool.
//
// One persistent CTA an SM, each with a share of the stream of pages (latent_units.cuh); a
// tile that is cut leaves unnormalised sums in the workspace, which a second kernel joins.
// More than 64 rows of one token, and large launches of prompt tokens, take tiles of 128
// rows on pairs of SMs (latent_pair.cu).
//
// Softmax: P = 2^(s scale log2(e) - ref).  P is rounded to bf16 and summed in float32,
// whose relative precision does not depend on the reference, so that need not be the
// maximum: it is 2^24 above the score of the row's first key, and is raised (to 2^24 above a
// page's maximum) only when a score exceeds it by 2^8, so that sums leave float32's range for
// latents beyond 2^119 / keys alone (from the score itself, with 2^32 above it: 2^95 / keys).
// The usual page needs no maximum across threads, only a vote.
//
// Warps: 0 loads (TMA), 1 issues the products, 2-5 do the softmax: warp w holds keys
// 16 (w % 4) .. + 15 of S^T and 32 lanes of each 128 numbers of O^T.
//
// A value that is not finite, at a key that some rows of a tile see and others do not,
// would reach all of them through 0 * NaN.  Key rows that no token of the tile sees are
// zeroed before they are values; a row whose output is not finite while its sum is, and
// which does not see such a key of the tile, computes again from its own (attend_again; the
// other roles' waits allow for the time, latent.cuh).
//
// Bound: HBM while all CTAs stream (64 rows of 32 heads, 512 to 8192 keys: 322 MB in 47 us, about
// the copy rate), then the start (9 us to the first value product), the tiles' ends and the
// join: 68.6 us, 4.7 TB/s.  (Prefetches into L2 ahead of the copies: 5 us more.)
#include "latent_units.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

constexpr int kThreads = 192;
constexpr int kSoftBar = 1;  // named barrier of the softmax warps

template <int NB, int N>
struct LatentSmem {
  static constexpr int kChunks = 2 * NB + 1;                 // 64 numbers of a row each; the last: the rotated ones
  static constexpr int kRg = kChunks * 1024;                 // eight keys: [chunk][8 rows of 128 bytes, swizzled]
  static constexpr int kStage = 8 * kRg;                     // a page
  static constexpr int kQ = kChunks * N * 128;
  static constexpr int kP = kPage * 128;
  static constexpr int kMisc = 2048;
  static constexpr int kBudget = 232448 - 1024 - kMisc - kQ - kP;
  static constexpr int kStages = kBudget / kStage < 4 ? kBudget / kStage : 4;
  static constexpr int kGroups = kPage / 16;                 // parts of a stage that are loaded and freed on their own
  static constexpr int kGroup = 2 * kRg;                     // 16 keys
  static constexpr size_t stage = 0;
  static constexpr size_t q = size_t(kStages) * kStage;
  static constexpr size_t p = q + kQ;
  static constexpr size_t bars = p + kP;
  // full[S], empty[S][groups], sfull[2], pfull, pvdone, qfull, qempty, fin
  static constexpr int kNumBars = kStages + kStages * kGroups + 7;
  static constexpr size_t keys = (bars + 8 * kNumBars + 15) & ~size_t(15);  // int2 a row
  static constexpr size_t alpha = keys + 8 * kLatentRows;      // factors of a raise; at the end 1 / sum
  static constexpr size_t ref = alpha + 4 * kLatentRows;
  static constexpr size_t misc = ref + 4 * kLatentRows;      // abort, tensor memory, beat, share
  static constexpr size_t end = misc + 256;
  static_assert(end - bars <= kMisc, "barriers and row data");
  static_assert(kStages >= 2, "stages");
  static constexpr size_t bytes = bars + kMisc + 1024;
  static constexpr uint32_t kColS = NB * N;                  // after O^T
  static constexpr uint32_t kCols = NB * N + 2 * N <= 64 ? 64 : NB * N + 2 * N <= 128 ? 128
                                  : NB * N + 2 * N <= 256 ? 256 : 512;
};

template <int NB, int N>
__global__ void __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap pmap,
                  const __grid_constant__ CUtensorMap rmap, const __grid_constant__ LatentParams p) {
  using L = LatentSmem<NB, N>;
  constexpr int kStages = L::kStages, kGroups = L::kGroups;
  constexpr int C = NB * 128;
  constexpr int kEnd = N < 32 ? N : 32;  // rows of a step of the epilogue
  constexpr int NX = N / 2;  // scores a softmax thread holds: N / 4 columns of two keys
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::bars);
  const uint32_t full = smem_addr(bars);                     // [stage]
  const uint32_t empty = full + 8 * kStages;                 // [stage][group]
  const uint32_t sfull = empty + 8 * kStages * kGroups;      // [2]
  const uint32_t pfull = sfull + 16, pvdone = pfull + 8, qfull = pvdone + 8, qempty = qfull + 8, fin = qempty + 8;
  int2* row_keys = reinterpret_cast<int2*>(smem + L::keys);  // keys that a row sees: [x, y)
  float* s_alpha = reinterpret_cast<float*>(smem + L::alpha);
  float* s_ref = reinterpret_cast<float*>(smem + L::ref);
  int* misc = reinterpret_cast<int*>(smem + L::misc);
  volatile int* abort_flag = misc;

  // the joining kernel may start: it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int team = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(full + 8 * i, 1);
    for (int i = 0; i < kStages; ++i) mbar_init(full + 8 * i, kGroups);
    mbar_init(pfull, 4);
    abort_flag[0] = abort_flag[kBeat] = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) tmem_alloc(smem_addr(misc + 1), L::kCols);

  // positions, rows and the table are read before the wait for the kernel before this one
  const Shares shares = count_shares<kThreads>(p, team, misc + 4);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(misc[1]));
  const Share* share = share_of(misc + 4);
  int t = share->t, j0 = share->j;
  long long left = static_cast<long long>(share->left);

  // what the kernel before this one on the stream writes is touched from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (shares.bad && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, shares.bad);
  if (tid == 0 && !p.whole) write_cut(p, team, t, left > 0 ? j0 : 0, shares.per);
  if (warp == 0) {
    // ============================== producer ==============================
    if (lane == 0) {
      int g = 0, issued = 0, units = 0;  // pages; parts of pages and query tiles whose copies were issued
      bool ok = true;
      auto load_q = [&](int t) {
        mbar_arrive_expect_tx(qfull, L::kQ);
        for (int c = 0; c < L::kChunks; ++c)
          tma_load_2d(smem_addr(smem + L::q) + c * (N * 128), &qmap, c * kBoxCols, t * p.heads, qfull);
        ++units;
      };
      if (left > 0) load_q(t);
      for (int u = 0; ok && left > 0; ++u) {
        const Unit un = unit_at(p, t);
        const int n = static_cast<int>(min(left, static_cast<long long>(un.np - j0)));
        const int32_t* trow = p.table + static_cast<long long>(max(un.row, 0)) * p.pages_per_row + un.first + j0;
        for (int i = 0; ok && i < n; ++i, ++g) {
          int page = un.row >= 0 ? trow[i] : 0;
          if (page < 0 || page >= p.num_pages) {
            if (p.status != nullptr && page_seen(p, t, un.nt, un.first + j0 + i)) atomicOr(p.status, LNK_DEV_BAD_PAGE);
            page = 0;  // (its keys are masked and its values zeroed)
          }
          const int st = g % kStages;
          const uint32_t dst = smem_addr(smem + L::stage) + st * L::kStage;
          for (int gr = 0; ok && gr < kGroups; ++gr) {
            const uint32_t fb = full + 8 * st;
            if (g >= kStages) ok = wait_with_beat(empty + 8 * (st * kGroups + gr), ((g / kStages) - 1) & 1, abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(fb, L::kGroup);
            if (p.rope_dim == 64) {
              tma_load_4d(dst + gr * L::kGroup, &pmap, 0, 0, 0, page * 8 + 2 * gr, fb);
            } else {
              for (int k = 2 * gr; k < 2 * gr + 2; ++k) {
                tma_load_4d(dst + k * L::kRg, &pmap, 0, 0, 0, page * 8 + k, fb);
                tma_load_2d(dst + k * L::kRg + 2 * NB * 1024, &rmap, C, page * kPage + k * 8, fb);
              }
            }
            ++issued;
          }
          if (ok && i == 0 && u > 0) {
            ok = wait_with_beat(qempty, (u - 1) & 1, abort_flag);
            if (ok) load_q(t);
          }
        }
        left -= n;
        t += un.nt;
        j0 = 0;
      }
      // do not leave while a copy may still land in this CTA's memory (pages whose every part
      // was asked for; a page that was given up halfway keeps its barrier to the limit)
      const int asked = (issued + kGroups - 1) / kGroups;
      for (int k = max(0, asked - kStages); k < asked; ++k) {
        const uint64_t t_0 = global_timer_ns();
        while (!mbar_try_wait(full + 8 * (k % kStages), (k / kStages) & 1) && global_timer_ns() - t_0 < kWaitLimitNs) {
        }
      }
      const uint64_t t_0 = global_timer_ns();
      while (units > 0 && !mbar_try_wait(qfull, (units - 1) & 1) && global_timer_ns() - t_0 < kWaitLimitNs) {
      }
    }
  } else if (warp == 1) {
    // =========================== products' issuer ===========================
    // The whole warp runs this, on values that are the same in all its threads.  The loops are
    // not unrolled: a launch starts with cold instruction caches, and 36 products in a row
    // took 14000 clocks the first time.
    constexpr uint32_t kIdS = umma_idesc_bf16(kPage, N, 0, 0);
    constexpr uint32_t kIdPV = umma_idesc_bf16(128, N, 1, 1);
    const uint64_t kdesc = umma_desc_sw128(smem_addr(smem + L::stage), 0, L::kRg);
    const uint64_t qdesc = umma_desc_sw128(smem_addr(smem + L::q), 0, 1024);
    const uint64_t vdesc = umma_desc_sw128(smem_addr(smem + L::stage), 1024, L::kRg);
    const uint64_t pdesc = umma_desc_sw128(smem_addr(smem + L::p), 0, 1024);
    const uint32_t k_lo = static_cast<uint32_t>(kdesc), k_hi = static_cast<uint32_t>(kdesc >> 32);
    const uint32_t q_lo = static_cast<uint32_t>(qdesc), q_hi = static_cast<uint32_t>(qdesc >> 32);
    const uint32_t v_lo = static_cast<uint32_t>(vdesc), v_hi = static_cast<uint32_t>(vdesc >> 32);
    const uint32_t p_lo = static_cast<uint32_t>(pdesc), p_hi = static_cast<uint32_t>(pdesc >> 32);
    // (reductions leave their results in uniform registers, which is where loop counters and
    // conditions must be for the products' operands to be there)
    auto uniform = [](int x) { return __reduce_max_sync(0xffffffffu, x); };
    auto done = [](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_test_wait(bar, parity)) != 0;
    };
    // S^T of page s and the value product of page v <= s are issued in whatever order they
    // become ready: neither waits for the other's data.
    int s = 0, v = 0, u = 0;           // next score page; next value page; unit of page s
    int ut = 0, un = 0, ui = 0;        // tokens and pages (of this share) of unit u, page s in it
    uint32_t first = 0u;               // bit s & 1: page s is its unit's first here
    int more = uniform(left > 0);      // page s exists
    if (more != 0) {
      const Unit x = unit_at(p, t);
      ut = x.nt;
      un = uniform(static_cast<int>(min(left, static_cast<long long>(x.np - j0))));
    }
    uint64_t t0 = 0;
    uint32_t idle = 0;
    while (more != 0 || v < s) {
      bool did = false;
      if (v < s && done(pfull, v & 1)) {
        tc_fence_after();
        const int st = v % kStages;
        const uint32_t vd = v_lo + ((st * L::kStage) >> 4);
        const uint32_t keep = first >> (v & 1) & 1u ? 0u : 1u;
#pragma unroll 1
        for (int kk = 0; kk < L::kGroups; ++kk) {
#pragma unroll
          for (int mb = 0; mb < NB; ++mb)
            umma_ss_warp(tmem + mb * N, vd + ((kk * L::kGroup + 2 * mb * 1024) >> 4), v_hi, p_lo + ((kk * 2048) >> 4), p_hi,
                         kIdPV, kk > 0 ? 1u : keep);
          umma_commit_warp(empty + 8 * (st * kGroups + kk));
        }
        umma_commit_warp(pvdone);
        ++v;
        did = true;
      }
      // (two score buffers: page s - 2 has been read once its value product was issued)
      if (more != 0 && s <= v + 1 && done(full + 8 * (s % kStages), (s / kStages) & 1) && (ui > 0 || done(qfull, u & 1))) {
        tc_fence_after();
        const uint32_t sc = tmem + L::kColS + (s & 1) * N;
        uint32_t kd = k_lo + (((s % kStages) * L::kStage) >> 4), qd = q_lo;
#pragma unroll 1
        for (int c = 0; c < 2 * NB; ++c, kd += 1024 >> 4, qd += (N * 128) >> 4) {
          umma_ss_warp(sc, kd, k_hi, qd, q_hi, kIdS, c > 0 ? 1u : 0u);
#pragma unroll
          for (int kk = 1; kk < 4; ++kk) umma_ss_warp(sc, kd + ((kk * 32) >> 4), k_hi, qd + ((kk * 32) >> 4), q_hi, kIdS, 1u);
        }
        umma_ss_warp(sc, kd, k_hi, qd, q_hi, kIdS, 1u);
        umma_ss_warp(sc, kd + (32 >> 4), k_hi, qd + (32 >> 4), q_hi, kIdS, 1u);
        if (p.rope_dim == 64) {
          umma_ss_warp(sc, kd + (64 >> 4), k_hi, qd + (64 >> 4), q_hi, kIdS, 1u);
          umma_ss_warp(sc, kd + (96 >> 4), k_hi, qd + (96 >> 4), q_hi, kIdS, 1u);
        }
        umma_commit_warp(sfull + 8 * (s & 1));
        first = (first & ~(1u << (s & 1))) | (ui == 0 ? 1u << (s & 1) : 0u);
        ++s;
        if (++ui == un) {  // the unit's last scores: its query rows may go
          umma_commit_warp(qempty);
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
    umma_commit_warp(fin);
    wait_with_beat(fin, 0, abort_flag);
    __syncwarp();
  } else {
    // ============================== softmax ===============================
    const int qt = warp & 3;
    const int sid = tid - 64;                 // 0 .. 127
    const int ka = qt * 16 + (lane >> 2);     // this thread's keys of a page: ka, ka + 8
    const int ca = 2 * (lane & 3);            // its columns: 8 i + ca, + 1
    const uint32_t lanes = static_cast<uint32_t>(qt * 32) << 16;
    float* scratch = reinterpret_cast<float*>(smem + L::p);  // [4][N], while no P is there
    const uint64_t scale2 = f32x2(p.scale_log2, p.scale_log2);
    bool ok = true;
    int g = 0;
    while (ok && left > 0) {
      const Unit un = unit_at(p, t);
      const int n = static_cast<int>(min(left, static_cast<long long>(un.np - j0)));
      const int nrows = un.nt * p.heads;  // at most N
      const int rowbase = t * p.heads;
      const bool direct = j0 == 0 && n == un.np;
      named_barrier_sync(kSoftBar, 128);  // (the unit before is done with the rows' data)
      // keys that each row sees (rows past the unit's: everything, nobody reads them)
      if (sid < N) {
        int lo = 0, hi = 0x7fffffff, row;
        if (sid < nrows) token_keys(p, t + sid / p.heads, row, lo, hi);
        row_keys[sid] = make_int2(lo, hi);
        s_ref[sid] = -INFINITY;  // the score of the row's first key, once it is known
      }
      named_barrier_sync(kSoftBar, 128);
      const int32_t* trow = p.table + static_cast<long long>(max(un.row, 0)) * p.pages_per_row;
      float nref[N / 4], l[N / 4];  // minus the reference (0 while there is none), this thread's part of the sum
      uint32_t unset = 0u;          // columns (bit) without a reference that see keys
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        const int col = 8 * (i >> 1) + ca + (i & 1);
        nref[i] = col < nrows ? 0.f : -INFINITY;  // (rows past the unit's have no weights, and nothing to raise)
        l[i] = 0.f;
        if (col < nrows && row_keys[col].y > row_keys[col].x) unset |= 1u << i;
      }
      bool force = true;            // some row has no reference yet (the same in every thread)
      for (int i = 0; i < n; ++i, ++g) {
        const int lp = un.first + j0 + i, kb = lp * kPage;
        const int page = un.row >= 0 ? trow[lp] : -1;
        const bool held = page >= 0 && page < p.num_pages;
        ok = __all_sync(0xffffffffu, wait_with_beat(sfull + 8 * (g & 1), (g >> 1) & 1, abort_flag));
        tc_fence_after();
        uint32_t r[NX];
        if (ok) {
          tmem_ld_16x256b(tmem + lanes + L::kColS + (g & 1) * N, r);
          tmem_ld_wait();
        }
        // (The paths off the usual page are kept short: their instructions are cold when they
        // are met, a line of them a few hundred clocks.)
        if (!(held && kb >= un.in_lo && kb + kPage <= un.in_hi)) {
          if (un.nt == 1 || !held) {  // one row of the table's keys for all columns
            const bool see0 = held && kb + ka >= un.kmin && kb + ka < un.kmax;
            const bool see8 = held && kb + ka + 8 >= un.kmin && kb + ka + 8 < un.kmax;
#pragma unroll
            for (int x = 0; x < NX; ++x)
              if (!(x & 2 ? see8 : see0)) r[x] = 0xFF800000u;
          } else {
#pragma unroll
            for (int x = 0; x < NX; x += 4) {
              const int4 k = *reinterpret_cast<const int4*>(row_keys + 2 * x + ca);  // of columns 2 x + ca, + 1
              const int key = kb + ka;
              if (key < k.x || key >= k.y) r[x] = 0xFF800000u;
              if (key < k.z || key >= k.w) r[x + 1] = 0xFF800000u;
              if (key + 8 < k.x || key + 8 >= k.y) r[x + 2] = 0xFF800000u;
              if (key + 8 < k.z || key + 8 >= k.w) r[x + 3] = 0xFF800000u;
            }
          }
        }
        if (force) {
          if (un.nt == 1 || p.window == 0) {  // the same first key for all rows
            const int first = max(un.kmin, kb) - kb;
            if (ka == first || ka + 8 == first) {
#pragma unroll
              for (int x = 0; x < N / 4; ++x) {
                const int at = (x >> 1) * 4 + (x & 1);
                s_ref[8 * (x >> 1) + ca + (x & 1)] = __uint_as_float(ka == first ? r[at] : r[at + 2]);
              }
            }
          } else {
#pragma unroll 1
            for (int col = 0; col < N; ++col) {
              // (the thread that holds the column's first key of this page)
              const int first = max(row_keys[col].x, kb) - kb - ka;
              if ((first == 0 || first == 8) && (col & 6) == ca) {
                float f = -INFINITY;
#pragma unroll
                for (int x = 0; x < NX; ++x)
                  if (8 * (x >> 2) + ca + (x & 1) == col && (x & 2 ? 8 : 0) == first) f = __uint_as_float(r[x]);
                s_ref[col] = f;
              }
            }
          }
          named_barrier_sync(kSoftBar, 128);
#pragma unroll
          for (int x = 0; x < N / 4; ++x) {
            const float f = s_ref[8 * (x >> 1) + ca + (x & 1)];
            if ((unset >> x & 1) && f > -INFINITY) {  // (a NaN score: the maximum of the others, below)
              nref[x] = fmaf(-f, p.scale_log2, -kAheadLog2);
              unset &= ~(1u << x);
            }
          }
        }
        float a[NX];
        float mx = -INFINITY;
        auto exponents = [&]() {
#pragma unroll
          for (int x = 0; x < NX; x += 2) {
            const int i0 = (x >> 2) * 2;
            f32x2_split(fma_f32x2(f32x2(__uint_as_float(r[x]), __uint_as_float(r[x + 1])), scale2,
                                  f32x2(nref[i0], nref[i0 + 1])),
                        a[x], a[x + 1]);
            mx = fmax3(mx, a[x], a[x + 1]);
          }
        };
        exponents();
        if (force) {
          // a column without a reference that sees a score all the same (its first one is -inf)
          if (unset != 0u) {
#pragma unroll
            for (int x = 0; x < NX; ++x)
              if ((unset >> ((x >> 2) * 2 + (x & 1)) & 1) && a[x] > -INFINITY) mx = INFINITY;
          }
          force = __any_sync(0xffffffffu, unset != 0u);
        }
        if (named_barrier_or(kSoftBar, 128, mx > kRaiseLog2 || !ok)) {
          // ---- references raised (or set) with the page's maximum ----
          if (g > 0 && ok) ok = __all_sync(0xffffffffu, wait_with_beat(pvdone, (g - 1) & 1, abort_flag));
          if (named_barrier_or(kSoftBar, 128, !ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int x = 0; x < N / 4; ++x) {
            const int at = (x >> 1) * 4 + (x & 1);
            float m = fmaxf(__uint_as_float(r[at]), __uint_as_float(r[at + 2]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (lane < 4) scratch[qt * N + 8 * (x >> 1) + ca + (x & 1)] = m;
          }
          named_barrier_sync(kSoftBar, 128);
          bool moved = false;
#pragma unroll
          for (int x = 0; x < N / 4; ++x) {
            const int col = 8 * (x >> 1) + ca + (x & 1);
            float m = fmaxf(fmaxf(scratch[col], scratch[N + col]), fmaxf(scratch[2 * N + col], scratch[3 * N + col]));
            float f = 1.f;
            if (m != -INFINITY) {
              m *= p.scale_log2;
              if (unset >> x & 1) {
                nref[x] = -m - kAheadLog2;
                unset &= ~(1u << x);
              } else if (m + nref[x] > kRaiseLog2) {
                f = ex2_approx((-m - kAheadLog2) - nref[x]);
                l[x] *= f;
                nref[x] = -m - kAheadLog2;
                moved = true;
              }
            }
            if (sid < 4) s_alpha[col] = f;
          }
          force = __any_sync(0xffffffffu, unset != 0u);
          moved = __any_sync(0xffffffffu, moved);
          named_barrier_sync(kSoftBar, 128);
          if (moved && i > 0) {
#pragma unroll 1
            for (int c = 0; c < NB * N; c += 16) {
              uint32_t v[16];
              tmem_ld16(tmem + lanes + c, v);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * s_alpha[(c + k) % N]);
              tmem_st16(tmem + lanes + c, v);
            }
            tmem_st_wait();
          }
          exponents();
        }
        // ---- P^T into shared memory, once the product before has read the last one ----
        if (g > 0) ok = __all_sync(0xffffffffu, wait_with_beat(pvdone, (g - 1) & 1, abort_flag));
        uint8_t* prow = smem + L::p + ka * 128 + (lane & 3) * 4;
#pragma unroll
        for (int x = 0; x < NX; x += 4) {
          const int i0 = x >> 1, chunk = x >> 2;
          const float e0 = ex2_approx(a[x]), e1 = ex2_approx(a[x + 1]);
          const float e2 = ex2_approx(a[x + 2]), e3 = ex2_approx(a[x + 3]);
          l[i0] += e0 + e2;
          l[i0 + 1] += e1 + e3;
          const int at = (chunk ^ (ka & 7)) << 4;
          *reinterpret_cast<uint32_t*>(prow + at) = pack_bf16x2(e0, e1);
          *reinterpret_cast<uint32_t*>(prow + 8 * 128 + at) = pack_bf16x2(e2, e3);
        }
        // ---- value rows that no token of the unit sees may hold anything: zero ----
        if (!(held && kb >= un.kmin && kb + kPage <= un.kmax)) {
          uint8_t* v = smem + L::stage + (g % kStages) * L::kStage;
          // rows [0, below) and [above, 64), 16 bytes of a row a thread (eight threads a line)
          const int below = held ? min(kPage, max(0, un.kmin - kb)) : kPage;
          const int above = held ? max(below, min(kPage, un.kmax - kb)) : kPage;
          const int out = below + kPage - above;
#pragma unroll 1
          for (int k = sid >> 3; k < out; k += 16) {
            const int key = k < below ? k : k - below + above;
            uint8_t* to = v + (key >> 3) * L::kRg + (key & 7) * 128 + (sid & 7) * 16;
#pragma unroll
            for (int c = 0; c < 2 * NB; ++c) *reinterpret_cast<uint4*>(to + c * 1024) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull);
      }
      // ---- the unit's end: sums joined, outputs or partial sums stored ----
      if (ok) ok = __all_sync(0xffffffffu, wait_with_beat(pvdone, (g - 1) & 1, abort_flag));
      if (named_barrier_or(kSoftBar, 128, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < N / 4; ++x) {
        float s = l[x];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane < 4) scratch[qt * N + 8 * (x >> 1) + ca + (x & 1)] = s;
        if (sid < 4) s_ref[8 * (x >> 1) + ca + (x & 1)] = nref[x];
      }
      named_barrier_sync(kSoftBar, 128);
      const size_t slot = direct ? 0 : static_cast<size_t>(2 * team + (j0 == 0 ? 1 : 0)) * p.slot_rows;
      if (sid < N) {
        const float s = (scratch[sid] + scratch[N + sid]) + (scratch[2 * N + sid] + scratch[3 * N + sid]);
        s_alpha[sid] = direct ? (s > 0.f ? 1.f / s : s) : (s == s ? 1.f : s);
        if (!direct) {
          p.ml[(slot + sid) * 2] = s == 0.f ? -INFINITY : -s_ref[sid];
          p.ml[(slot + sid) * 2 + 1] = s;
        }
      }
      named_barrier_sync(kSoftBar, 128);
      uint32_t odd = 0u;  // bits 15 and 31: an element is not finite
      if (direct) {
        // Numbers lane / 4 (+ 8, 16, 24) of two rows a thread, packed and transposed in blocks of
        // eight rows and eight numbers; then four lanes trade their pieces, so that each stores
        // 16 bytes of a row: 64 bytes of eight rows a store.
#pragma unroll 1
        for (int mb = 0; mb < NB; ++mb) {
#pragma unroll 1
          for (int c0 = 0; c0 < N && c0 < nrows; c0 += 8) {
            uint32_t v[4], w[4], m[4];
            tmem_ld_16x256b(tmem + lanes + mb * N + c0, v);
            tmem_ld_16x256b(tmem + lanes + (16u << 16) + mb * N + c0, w);
            tmem_ld_wait();
            const float f0 = s_alpha[c0 + ca], f1 = s_alpha[c0 + ca + 1];
            auto piece = [&](uint32_t x, uint32_t y) {
              return movmatrix_trans(pack_bf16x2(f0 == 0.f ? 0.f : __uint_as_float(x) * f0, f1 == 0.f ? 0.f : __uint_as_float(y) * f1));
            };
            m[0] = piece(v[0], v[1]);
            m[1] = piece(v[2], v[3]);
            m[2] = piece(w[0], w[1]);
            m[3] = piece(w[2], w[3]);
#pragma unroll
            for (int k = 0; k < 4; ++k) odd |= (m[k] & 0x7F807F80u) + 0x00800080u;
            // lane l of four: piece l of each lane's four
#pragma unroll
            for (int s = 1; s < 4; s <<= 1) {
              const bool up = (lane & s) != 0;
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k & s) continue;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? m[k] : m[k | s], s);
                if (up) m[k] = got;
                else m[k | s] = got;
              }
            }
            const int rr = c0 + (lane >> 2);
            if (rr < nrows)
              *reinterpret_cast<uint4*>(p.out + static_cast<size_t>(rowbase + rr) * C + mb * 128 + qt * 32 + (lane & 3) * 8) =
                  make_uint4(m[0], m[1], m[2], m[3]);
          }
        }
      } else {
        // a lane holds one number of every row: 128 bytes of a row a store
#pragma unroll 1
        for (int c = 0; c < NB * N; c += kEnd) {
          const int mb = c / N, c0 = c % N, dim = mb * 128 + qt * 32 + lane;
          if (c0 >= nrows) continue;
          uint32_t v[kEnd];
          if constexpr (kEnd == 32) tmem_ld32(tmem + lanes + c, v);
          else tmem_ld16(tmem + lanes + c, v);
          tmem_ld_wait();
          const bool whole = c0 + kEnd <= nrows;
          float* o = p.o + (slot + c0) * C + dim;
#pragma unroll
          for (int k = 0; k < kEnd; ++k) {
            if (whole || c0 + k < nrows) {
              o[k * C] = __uint_as_float(v[k]);
              odd |= ((v[k] >> 16 & 0x7F80u) + 0x0080u) & 0x8000u;
            }
          }
        }
      }
      if (__any_sync(0xffffffffu, (odd & 0x80008000u) != 0u)) {
        const int w = p.latent_dim + p.rope_dim;
        const int seg_lo = max(un.kmin, (un.first + j0) * kPage), seg_hi = min(un.kmax, (un.first + j0 + n) * kPage);
        int in_lo = 0, in_hi = 0x7fffffff;  // keys that every row with keys sees
        for (int rr = lane; rr < nrows; rr += 32) {
          if (row_keys[rr].y <= row_keys[rr].x) continue;
          in_lo = max(in_lo, row_keys[rr].x);
          in_hi = min(in_hi, row_keys[rr].y);
        }
        const int2 bad_keys = odd_keys<false>(p, trow, seg_lo, seg_hi, __reduce_max_sync(0xffffffffu, in_lo),
                                       __reduce_min_sync(0xffffffffu, in_hi), abort_flag);
#pragma unroll 1
        for (int rr = 0; rr < nrows; ++rr) {
          if (s_alpha[rr] != s_alpha[rr]) continue;  // (a sum that is NaN is the row's own: all of it is)
          // (so is what is not finite of a row that sees all such keys; one that sees nothing gets its zeros)
          if (row_keys[rr].y > row_keys[rr].x && row_keys[rr].x <= bad_keys.x && row_keys[rr].y > bad_keys.y) continue;
          bool bad = false;
#pragma unroll 1
          for (int mb = 0; mb < NB; ++mb) {
            uint32_t v[16];
            tmem_ld16(tmem + lanes + mb * N + (rr & ~15), v);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (k == (rr & 15)) bad |= (__float_as_uint(__uint_as_float(v[k]) * s_alpha[rr]) & 0x7F800000u) == 0x7F800000u;
          }
          if (!__any_sync(0xffffffffu, bad)) continue;
          __syncwarp();  // (other lanes stored what is stored again)
          float acc[NB];
          attend_again<NB, 128, false>(p, p.q + static_cast<size_t>(rowbase + rr) * w, trow, max(row_keys[rr].x, seg_lo),
                            min(row_keys[rr].y, seg_hi), s_ref[rr], qt * 32 + lane, acc, abort_flag);
#pragma unroll
          for (int mb = 0; mb < NB; ++mb) {
            const int dim = mb * 128 + qt * 32 + lane;
            if (direct)
              p.out[static_cast<size_t>(rowbase + rr) * C + dim] =
                  static_cast<uint16_t>(pack_bf16x2(acc[mb] * s_alpha[rr], 0.f));
            else
              p.o[(slot + rr) * C + dim] = acc[mb];
          }
        }
      }
      tc_fence_before();
      left -= n;
      t += un.nt;
      j0 = 0;
    }
    if (!ok) *abort_flag = 1;
  }
  __syncwarp();
  if (*abort_flag && lane == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, L::kCols);
}

template <int NB, int N>
cudaError_t launch_t(const CUtensorMap& qmap, const CUtensorMap& pmap, const CUtensorMap& rmap, const LatentParams& p, cudaStream_t stream) {
  const int bytes = static_cast<int>(LatentSmem<NB, N>::bytes);
  cudaError_t err = set_max_dynamic_smem(reinterpret_cast<const void*>(latent_kernel<NB, N>), bytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.teams));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  err = cudaLaunchKernelEx(&cfg, latent_kernel<NB, N>, qmap, pmap, rmap, p);
  if (err != cudaSuccess) return err;
  return launch_latent_join(p, stream);
}

}  // namespace

cudaError_t launch_latent_attn(const CUtensorMap& qmap, const CUtensorMap& pmap, const CUtensorMap& rmap, const LatentParams& p,
                               cudaStream_t stream) {
  switch (p.latent_dim / 128 * 100 + p.tile_rows) {
    case 116: return launch_t<1, 16>(qmap, pmap, rmap, p, stream);
    case 132: return launch_t<1, 32>(qmap, pmap, rmap, p, stream);
    case 164: return launch_t<1, 64>(qmap, pmap, rmap, p, stream);
    case 216: return launch_t<2, 16>(qmap, pmap, rmap, p, stream);
    case 232: return launch_t<2, 32>(qmap, pmap, rmap, p, stream);
    case 264: return launch_t<2, 64>(qmap, pmap, rmap, p, stream);
    case 316: return launch_t<3, 16>(qmap, pmap, rmap, p, stream);
    case 332: return launch_t<3, 32>(qmap, pmap, rmap, p, stream);
    case 364: return launch_t<3, 64>(qmap, pmap, rmap, p, stream);
    case 416: return launch_t<4, 16>(qmap, pmap, rmap, p, stream);
    case 432: return launch_t<4, 32>(qmap, pmap, rmap, p, stream);
    case 464: return launch_t<4, 64>(qmap, pmap, rmap, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
