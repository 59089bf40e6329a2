// How a latent attention launch's work is laid out: tiles of query rows that see one table
// row (units), their pages laid end to end in one stream, and the teams' equal shares of it.
// A unit is one decode row's token, or a run of prompt tokens of one table row that fit a
// tile together; with more heads than a tile has rows, each of the team's CTAs (or pairs)
// takes a block of heads over the same pages.
#pragma once

#include "latent.cuh"

namespace lnk {
namespace {

struct Share {
  unsigned long long left;  // pages of this team's share
  int t, j;                 // its first unit (that one's first token) and first page in it
};

struct Shares {
  long long per;  // pages of a share
  int bad;        // device status bits of this thread's tokens
};

struct Unit {
  int nt, row;        // tokens; table row (-1: nothing to see)
  int kmin, kmax;     // keys that some token sees
  int in_lo, in_hi;   // keys that every token sees
  int first, np;      // first page; pages (one at least)
};

__device__ __forceinline__ int token_keys(const LatentParams& p, int t, int& row, int& lo, int& hi) {
  int pos;
  if (t < p.P) {
    row = p.rows[t];
    pos = p.positions[t];
  } else {
    row = t - p.P;
    pos = p.step_positions[t - p.P];
  }
  lo = hi = 0;
  if (pos < 0) return 0;
  if (row < 0 || row >= p.num_rows) return LNK_DEV_BAD_ROW;
  if (pos >= p.pages_per_row * kPage) return LNK_DEV_BAD_POSITION;
  lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  hi = pos + 1;
  return 0;
}

__device__ __forceinline__ bool unit_starts(const LatentParams& p, int t) {
  return t >= p.P || p.tile_tokens == 1 || t % p.tile_tokens == 0 || p.rows[t] != p.rows[t - 1];
}

__device__ __forceinline__ Unit unit_at(const LatentParams& p, int t) {
  Unit u;
  u.nt = 0;
  u.row = -1;
  u.kmin = 0x7fffffff;
  u.kmax = 0;
  u.in_lo = 0;
  u.in_hi = 0x7fffffff;
  const int end = t < p.P ? min(p.P, (t / p.tile_tokens + 1) * p.tile_tokens) : t + 1;
  int row0 = 0;
  for (int s = t; s < end; ++s) {
    int row, lo, hi;
    token_keys(p, s, row, lo, hi);
    if (s == t) row0 = row;
    else if (row != row0) break;
    ++u.nt;
    u.in_lo = max(u.in_lo, lo);
    u.in_hi = min(u.in_hi, hi);
    if (hi > lo) {
      u.row = row;
      u.kmin = min(u.kmin, lo);
      u.kmax = max(u.kmax, hi);
    }
  }
  if (u.row < 0) u.kmin = 0;
  u.first = u.kmin / kPage;
  u.np = u.row < 0 ? 1 : (u.kmax - 1) / kPage - u.first + 1;
  return u;
}

// Whether a token of the unit that starts at t sees a key of the row's page lp: only then must the
// table name one (between the windows of tokens far apart lie pages that nobody needs).
__device__ __noinline__ bool page_seen(const LatentParams& p, int t, int nt, int lp) {
#pragma unroll 1
  for (int s = t; s < t + nt; ++s) {
    int row, lo, hi;
    token_keys(p, s, row, lo, hi);
    if (hi > lo && lo / kPage <= lp && lp <= (hi - 1) / kPage) return true;
  }
  return false;
}

// The first key from `from` on (to `to`, exclusive, in steps of +1 or -1) whose latent has a
// number that is not finite, or -1.  The whole warp.
template <bool kPair>
__device__ __noinline__ int odd_key(const LatentParams& p, const int32_t* trow, int from, int to, int step, volatile int* abort) {
  const int w = p.latent_dim + p.rope_dim, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int key = from; key != to; key += step) {
    if (key % kPage == 0) beat<kPair>(abort);
    const int page = trow[key / kPage];
    if (page < 0 || page >= p.num_pages) continue;
    const uint16_t* c = p.pool + (static_cast<size_t>(page) * kPage + key % kPage) * w;
    uint32_t odd = 0u;
#pragma unroll 1
    for (int e = lane * 8; e < p.latent_dim; e += 256) odd |= odd_halves(*reinterpret_cast<const uint4*>(c + e));
    if (__any_sync(0xffffffffu, odd != 0u)) return key;
  }
  return -1;
}

// The keys of [lo, hi) that rows which all see [in_lo, in_hi) may not see and that hold numbers
// which are not finite: a row that starts behind x or ends at or before y has some of them.
template <bool kPair>
__device__ __forceinline__ int2 odd_keys(const LatentParams& p, const int32_t* trow, int lo, int hi, int in_lo, int in_hi,
                                         volatile int* abort) {
  const int a = min(in_lo, hi), b = max(in_hi, lo);
  const int x = lo < a ? odd_key<kPair>(p, trow, lo, a, 1, abort) : -1;
  return make_int2(x < 0 ? 0x7fffffff : x, b < hi ? odd_key<kPair>(p, trow, hi - 1, b - 1, -1, abort) : -1);
}

// One row's sums over its own visible keys [lo, hi), relative to the reference that its softmax
// used: number d + STEP i of the latent in acc[i].  The whole warp: a key a lane for the
// scores, the numbers of a key over the lanes for the sums.
template <int NV, int STEP, bool kPair>
__device__ __noinline__ void attend_again(const LatentParams& p, const uint16_t* q, const int32_t* trow, int lo, int hi,
                                          float nref, int d, float (&acc)[NV], volatile int* abort) {
  const int w = p.latent_dim + p.rope_dim, lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.f;
#pragma unroll 1
  for (int key0 = lo; key0 < hi; key0 += 32) {
    beat<kPair>(abort);
    const int key = key0 + lane;
    const int page = key < hi ? trow[key / kPage] : -1;
    const bool here = page >= 0 && page < p.num_pages;
    const uint16_t* k = p.pool + (here ? (static_cast<size_t>(page) * kPage + key % kPage) * w : 0);
    float e = 0.f;
    if (here) {
      float s = 0.f;
#pragma unroll 4
      for (int i = 0; i < w; i += 8) s = dot8(*reinterpret_cast<const uint4*>(q + i), *reinterpret_cast<const uint4*>(k + i), s);
      e = exp2f(fmaf(s, p.scale_log2, nref));
    }
    unsigned todo = __ballot_sync(0xffffffffu, here);
#pragma unroll 2
    while (todo != 0u) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const float f = __shfl_sync(0xffffffffu, e, src);
      const uint16_t* v = reinterpret_cast<const uint16_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(k), src)) + d;
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = fmaf(f, bf16_at(v + STEP * i), acc[i]);
    }
  }
}

// Counts the units' pages and finds this team's share: all threads of the CTA, each with a
// range of tokens.  mem: 40 ints of shared memory, 8-byte aligned; share_of(mem) is the
// result, after a barrier of the CTA.
__device__ __forceinline__ const Share* share_of(const int* mem) { return reinterpret_cast<const Share*>(mem + 20); }

template <int kThreads>
__device__ __forceinline__ Shares count_shares(const LatentParams& p, int team, int* mem) {
  constexpr int kWarps = kThreads / 32;
  static_assert(kWarps <= 10, "shared memory of the count");
  long long* scan = reinterpret_cast<long long*>(mem);   // [kWarps]
  Share* share = reinterpret_cast<Share*>(mem + 20);
  int* longest = mem + 24;                               // [kWarps]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    share->t = 0x7fffffff;
    share->j = 0;
    share->left = 0ull;
  }
  const int span = (p.T + kThreads - 1) / kThreads;
  const int ta = min(p.T, tid * span), tb = min(p.T, ta + span);
  int bad = 0, most = 0;
  long long mine = 0;
  for (int t = ta; t < tb; ++t) {
    int row, lo, hi;
    bad |= token_keys(p, t, row, lo, hi);
    if (unit_starts(p, t)) {
      const int np = unit_at(p, t).np;
      mine += np;
      most = max(most, np);
    }
  }
  most = __reduce_max_sync(0xffffffffu, most);
  long long before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) scan[warp] = before;
  if (lane == 0) longest[warp] = most;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
    most = max(most, longest[w]);
  }
  before -= mine;
  const long long per = max(1ll, (total + p.teams - 1) / p.teams);
  const long long start = team * per;
  // Units of few pages (or far fewer than a share) stay whole: a team takes those whose first
  // page lies in its share.
  const bool whole = p.whole || most <= max(static_cast<long long>(kWholePages), per / 8);
  if (before < start + per && before + mine > start) {
    long long at = before;
    for (int t = ta; t < tb && at < start + per; ++t) {
      if (!unit_starts(p, t)) continue;
      const int np = unit_at(p, t).np;
      if (whole) {
        if (at >= start) {
          atomicMin(&share->t, t);
          atomicAdd(&share->left, static_cast<unsigned long long>(np));
        }
      } else if (at <= start && start < at + np) {
        share->t = t;
        share->j = static_cast<int>(start - at);
        share->left = static_cast<unsigned long long>(min(per, total - start));
        break;
      }
      at += np;
    }
  }
  return {per, bad};
}

// What the joining kernel needs to know of the unit in which a share starts (j0 pages into it).
__device__ __forceinline__ void write_cut(const LatentParams& p, int team, int t, int j0, long long per) {
  LatentCut cut;
  cut.t0 = t;
  cut.nt = cut.np = 0;
  cut.j0 = j0;
  cut.per = per;
  cut.pad = 0;
  if (j0 > 0) {
    const Unit u = unit_at(p, t);
    cut.nt = u.nt;
    cut.np = u.np;
  }
  p.cuts[team] = cut;
}

}  // namespace
}  // namespace lnk
