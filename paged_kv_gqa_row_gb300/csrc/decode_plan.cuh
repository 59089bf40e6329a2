// How a decode launch's work is laid out: each (row, kv head) pair is a run of
// page-heads, and the runs of all pairs, (b, h) with h fastest, are laid end to
// end in one stream that the CTAs cut into chunks (decode.cu, decode4.cu).
#pragma once

#include "common.cuh"

namespace lnk {
namespace {

__device__ __forceinline__ int visible_pages(int pos, int window, int pages_per_row, int* bad) {
  if (pos < 0) return 0;
  if (pos >= pages_per_row * kPage) {
    *bad = LNK_DEV_BAD_POSITION;
    return 0;
  }
  const int lo = window > 0 ? max(0, pos - window + 1) : 0;
  return pos / kPage - lo / kPage + 1;
}

// Where page-head `gi` of the flattened stream lies, and the per-pair values
// the producer needs (computed once per pair, not per page).
struct Cursor {
  int b, h, j, np, pos, lo, first_page;
  int seg, c0, nseg, whole;
  const int* trow;
};

__device__ __forceinline__ void locate(Cursor& c, long long gi, const int* pref, const DecodeParams& p,
                                       long long start, long long end, long long per, long long chunk) {
  int lo_b = 0, hi_b = p.B - 1;  // largest b with hkv * pref[b] <= gi
  while (lo_b < hi_b) {
    const int mid = (lo_b + hi_b + 1) >> 1;
    if (static_cast<long long>(pref[mid]) * p.hkv <= gi) lo_b = mid; else hi_b = mid - 1;
  }
  c.b = lo_b;
  c.np = pref[c.b + 1] - pref[c.b];
  const long long rem = gi - static_cast<long long>(pref[c.b]) * p.hkv;
  c.h = static_cast<int>(rem / c.np);
  c.j = static_cast<int>(rem % c.np);
  c.pos = p.positions[c.b];
  c.lo = p.window > 0 ? max(0, c.pos - p.window + 1) : 0;
  c.first_page = c.lo / kPage;
  c.trow = p.table + static_cast<long long>(c.b) * p.pages_per_row;
  const long long pair_start = gi - c.j;
  const long long pair_end = pair_start + c.np;
  c.whole = pair_start >= start && pair_end <= end;
  c.c0 = static_cast<int>(pair_start / per);
  c.nseg = static_cast<int>((pair_end - 1) / per) - c.c0 + 1;
  c.seg = c.b * p.hkv + c.h + static_cast<int>(chunk);
}

}  // namespace
}  // namespace lnk
