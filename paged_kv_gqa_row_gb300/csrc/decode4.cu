// Paged split-KV decode attention over 4-bit pools (LNK_KV_E2M1).
//
// The work decomposition, the partial results of cut pairs and their merge are
// decode.cu's (decode_plan.cuh).  What differs is the CTA's inside, because a
// page of one head is only 36 D bytes of K and of V: at the rate HBM delivers
// them, an SM has about 390 cycles for the 16384 elements of a page's K and V
// (D = 128).  So the instructions spent per page decide, every scheduler needs
// as many warps at work as registers allow, and whatever is paid per page is
// paid by one warp per page:
//  * warps 0 .. kWarps - 1, consumers: the CTA's chunk of the stream is cut into
//    one run of pages per warp, and a warp works through its run alone, page
//    after page (64 keys), with an online softmax of its own.  A pair that lies
//    inside a run is finished there, in registers.  What a run has of a longer
//    pair is a piece: its state waits in shared memory until all warps are done,
//    and then the whole CTA merges the pieces of each pair, in their order.
//    (Dealing the pages of a pair out to all warps instead took a merge of 11
//    states per pair, by one warp, while the others waited: 121 us against 65 for
//    the example below.)
//  * a producer warp, whose lane w feeds consumer w: the lanes walk their
//    consumers' runs side by side (page table, masks) and load each page's K and
//    V, two contiguous blocks of 36 D bytes, into the consumer's own ring of
//    three blocks (K, V, K, V, ... in turn).  One lane for all consumers took
//    about 1100 cycles a page and held the kernel at 4.2 TB/s.
// One CTA per SM: its consumers and the producer take the whole register file.
// 64 rows of 512 to 8192 keys, 32 query heads on 8, D = 128: 62 us, 5.2 TB/s (169 us
// on bf16 pools).  A stream of the same blocks without arithmetic takes 53 us; the
// rest is the start, and at the end the merges of pieces and of cut pairs (6 to 9
// us).  Fifteen consumers with two blocks each, the next page's values loaded ahead,
// and packed half arithmetic were no faster.  D = 96 pays 1031 warp instructions a page
// where D = 128 pays 1057 for a third more bytes (narrower loads, two sets of value
// scales, a second product path): 32 rows of windows of 2047, a head per query head,
// stream 4.9 TB/s between the ends, the above 6.05.
//
// Arithmetic.  A code times its block's E4M3 scale has at most five significant
// bits and lies in f16's range (2^-10 .. 2688), so the converted keys and values
// are exact; the query is rounded to f16 (exact in the range the header states),
// the probabilities to f16, and all sums are float32.  Probabilities are relative to
// 2^-14 of the largest, so that the largest is 2^14 in f16: those down to 2^-28 of it
// are rounded to 2^-11 relative, and what smaller ones lose is below 2^-39 of it each.
// (The factor is in the denominator too.)
//
// Fragments (mma m16n8k16, lane = 4 r + c).  The order of the contraction index
// and of the output rows is free as long as both operands agree, so that every
// lane reads whole words of codes and needs few scales:
//  * S^T = K Q^T: lane (r, c) holds key perm(r) + 8 i (i = 0 .. 7, perm(r) =
//    (r >> 1) + 4 (r & 1)) and dimensions c D/4 .. (c + 1) D/4 - 1: one block
//    (two for D > 64), whose scales for its 8 keys are every other byte of a
//    16-byte load;
//  * O^T += V^T P^T: lane (r, c) holds keys c + 4 i (i = 0 .. 15) and a word of
//    dimensions around r (16 r .. for D = 128): its block's 16 scales are one
//    16-byte load, already in pairs.  Two keys' words are interleaved nibble by
//    nibble (four logic operations for eight pairs), after which a byte holds
//    one dimension of two keys, which is what the conversion takes.
// Masked keys: their scores become -inf and their value scales zero, so whatever
// the page holds there (a NaN scale too) adds nothing: codes are always finite.
//
// Sources: as decode.cu; the 4-bit format is this library's (lnk_attn_desc).
#include "common.cuh"
#include "decode_plan.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

constexpr int kWarps = 11;  // consumer warps; with the producer 12: 3 per scheduler at 168 registers
constexpr int kProducerWarp = kWarps;
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kRing = 3;    // blocks (a page's K, or its V) in a consumer's ring
// Page records per consumer.  A page's record is read until its piece is dealt
// with, after its blocks were freed; page ip + 4 is recorded only once page ip +
// 2 has been used up.
constexpr int kPages = 4;
constexpr int kEnd = 1;
constexpr int kFirst = 2;  // the piece's first page
constexpr int kLast = 4;   // the piece's last page
constexpr int kWhole = 8;  // the piece is its whole pair
constexpr int kRunEnd = 16;  // the run's last page
constexpr int kPieces = 2 * kWarps;  // a run's first and last piece
constexpr float kHeadroomLog2 = 14.f;  // the largest probability is 2^14 (f16 ends at 65504)

struct Page {
  int b, h, klo, khi, flags;
};

template <int D>
struct Smem {
  static constexpr int kBlock = 36 * D;               // K or V of a page
  static constexpr int kOStride = D + 4;              // padded row of a warp's state
  static constexpr int kStateFloats = kMaxGroup * kOStride;
  static constexpr size_t ring = 0;                                                  // [kWarps][kRing][kBlock]
  // States of a run's first piece; that of its last piece goes into the warp's
  // ring, which is free by then.
  static constexpr size_t state = ring + size_t(kWarps) * kRing * kBlock;            // [kWarps][kMaxGroup][kOStride]
  static constexpr size_t smax = state + size_t(kWarps) * kStateFloats * 4;          // [kPieces][kMaxGroup]
  static constexpr size_t ssum = smax + size_t(kPieces) * kMaxGroup * 4;
  static constexpr size_t bars = ssum + size_t(kPieces) * kMaxGroup * 4;             // full, empty: [kWarps][kRing]
  static constexpr size_t info = bars + size_t(2 * kWarps * kRing) * sizeof(uint64_t);  // [kWarps][kPages]
  static constexpr size_t pair = info + size_t(kPages * kWarps) * sizeof(Page);      // [kPieces]: b * Hkv + h, or -1
  static constexpr size_t misc = pair + kPieces * 4;  // abort, longest pair, warp sums, last arrivals [2], shared pairs [2][3]
  static constexpr size_t pref = misc + (2 + kWarps + 1 + 2 + 6) * 4;
  static_assert(kStateFloats * 4 <= kRing * kBlock, "a state fits the ring");
  static_assert(kBlock % 128 == 0 && state % 16 == 0 && bars % 8 == 0, "alignment of copies, states and barriers");
  static size_t bytes(int B) { return pref + size_t(B + 1) * 4 + 128; }  // + alignment slack
  static_assert(pref + size_t(kMaxDecodeRows + 1) * 4 + 128 <= 227 * 1024, "one CTA's shared memory");
};

__device__ __forceinline__ uint32_t low2(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t h) { return __byte_perm(h, h, 0x3232); }

// The bits of a where m has ones, of b elsewhere (one operation).
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t m) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xE4;" : "=r"(d) : "r"(a), "r"(b), "r"(m));
  return d;
}

// Byte order of eight codes of two keys, one dimension of both per byte: the
// even dimensions' codes (low four bits of a and of b) ...
__device__ __forceinline__ uint32_t mix_even(uint32_t a, uint32_t b) {
  return select_bits(a, b << 4, 0x0F0F0F0Fu);
}
// ... and the odd ones'.
__device__ __forceinline__ uint32_t mix_odd(uint32_t a, uint32_t b) {
  return select_bits(a >> 4, b, 0x0F0F0F0Fu);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) decode4_kernel(const DecodeParams p) {
  using L = Smem<D>;
  constexpr int KS = D / 16;  // k-steps of Q.K, d-tiles of P.V, blocks of a row
  constexpr int KW = D / 32;  // words of a key row per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::bars);  // [kWarps][kRing]
  uint64_t* empty_bar = full_bar + kWarps * kRing;
  Page* info = reinterpret_cast<Page*>(smem + L::info);
  int* piece_pair = reinterpret_cast<int*>(smem + L::pair);
  float* state = reinterpret_cast<float*>(smem + L::state);
  float* smax = reinterpret_cast<float*>(smem + L::smax);
  float* ssum = reinterpret_cast<float*>(smem + L::ssum);
  int* misc = reinterpret_cast<int*>(smem + L::misc);  // [0] abort, [1] longest pair, [2..13] warp sums of the scan
  int* arrived_last = misc + 2 + kWarps + 1;           // [2]: this CTA is the last of its first / last pair's
  int* shared = arrived_last + 2;                      // [2][3]: the chunk's first and last pair (below)
  volatile int* abort_flag = misc;
  int* pref = reinterpret_cast<int*>(smem + L::pref);

  // Let the next kernel on the stream start its own prologue (it waits for
  // this grid before it reads the output).
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int B = p.B;
  const int G = p.group;

  if (tid < kWarps * kRing) {
    mbar_init(smem_addr(full_bar + tid), 1);
    mbar_init(smem_addr(empty_bar + tid), 1);
    if (tid < kPieces) piece_pair[tid] = -1;
    if (tid == 0) {
      misc[0] = 0;
      misc[1] = 0;
    }
    fence_mbarrier_init();
  }

  // ---- per-row visible page counts and their prefix sums (all threads) ----
  {
    const int chunk = (B + kThreads - 1) / kThreads;
    const int r0 = min(B, tid * chunk), r1 = min(B, r0 + chunk);
    int bad = 0, run = 0, longest = 0;
    for (int b = r0; b < r1; ++b) {
      const int np = visible_pages(p.positions[b], p.window, p.pages_per_row, &bad);
      longest = max(longest, np);
      run += np;
      pref[b + 1] = run;
    }
    if (bad && p.status != nullptr && blockIdx.x == 0) atomicOr(p.status, bad);
    int incl = run;  // inclusive scan of the per-thread totals across the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) misc[2 + warp] = incl;
    __syncthreads();  // (also orders misc[1] = 0 above before the maxima below)
    if (longest > 0) atomicMax(misc + 1, longest);
    int off = incl - run;
    for (int w = 0; w < warp; ++w) off += misc[2 + w];
    for (int b = r0; b < r1; ++b) pref[b + 1] += off;
    if (tid == 0) pref[0] = 0;
    __syncthreads();
  }

  const long long total = static_cast<long long>(pref[B]) * p.hkv;
  const long long pairs = static_cast<long long>(B) * p.hkv;
  // At most one pair per CTA, none longer than twice a CTA's share: each chunk
  // is one whole pair (no partial results, no merges).
  const bool pair_chunks = pairs <= gridDim.x && 2 * ((total + gridDim.x - 1) / gridDim.x) >= misc[1];
  const long long per = (total + gridDim.x - 1) / gridDim.x;  // chunk size
  const long long nchunks = pair_chunks ? pairs : (per > 0 ? (total + per - 1) / per : 0);
  const long long chunk = blockIdx.x;

  long long start, end;  // the chunk's page-heads
  if (pair_chunks) {
    const int b = static_cast<int>(chunk / p.hkv), h = static_cast<int>(chunk % p.hkv);
    const int np = chunk < nchunks ? pref[b + 1] - pref[b] : 0;
    start = chunk < nchunks ? static_cast<long long>(pref[b]) * p.hkv + static_cast<long long>(h) * np : 0;
    end = start + np;
  } else {
    start = chunk * per;
    end = min(total, start + per);
  }

  // rows with nothing to attend to get a zero output, once the previous kernel
  // on the stream is done
  auto zero_rows = [&]() {
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      if (pref[b + 1] == pref[b]) {
        uint32_t* o = reinterpret_cast<uint32_t*>(p.out + static_cast<size_t>(b) * p.hq * D);
        for (int i = tid; i < p.hq * D / 2; i += kWarps * 32) o[i] = 0u;
      }
    }
  };
  if (start >= end) {
    if (warp != kProducerWarp) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      zero_rows();
    }
    return;
  }
  const long long n = end - start;
  // warp w's run of page-heads
  auto run_begin = [&](int w) { return start + n * w / kWarps; };

  // The pairs of the chunk's first and last page-head, where other chunks have
  // pages of them too: pair, first chunk, chunks (0: not shared).
  if (tid < 2) {
    Cursor e;
    locate(e, tid == 0 ? start : end - 1, pref, p, start, end, per, chunk);
    const int q = e.b * p.hkv + e.h;
    shared[tid * 3] = q;
    shared[tid * 3 + 1] = e.c0;
    shared[tid * 3 + 2] = e.whole || (tid == 1 && end - 1 - e.j <= start) ? 0 : e.nseg;
  }

  if (warp == kProducerWarp) {
    // ============================== producer ==============================
    const int w = min(lane, kWarps - 1);
    uint64_t* full = full_bar + w * kRing;
    uint64_t* empty = empty_bar + w * kRing;
    const long long rb = run_begin(w), re = run_begin(w + 1);
    long long gi = rb;
    Cursor cur;
    int entry = 0;  // the page table's entry for page-head gi
    if (gi < re) {
      locate(cur, gi, pref, p, start, end, per, chunk);
      entry = cur.trow[cur.first_page + cur.j];
    }
    // on to the next head or row (the lanes cross pairs one at a time, so this
    // has to be short)
    auto next_pair = [&]() {
      cur.j = 0;
      if (++cur.h < p.hkv) return;
      cur.h = 0;
      ++cur.b;
      if (pref[cur.b + 1] == pref[cur.b]) {  // rows without pages: the first one that has some
        int lo = cur.b + 1, hi = B - 1;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (pref[mid + 1] > pref[cur.b]) hi = mid; else lo = mid + 1;
        }
        cur.b = lo;
      }
      cur.np = pref[cur.b + 1] - pref[cur.b];
      cur.pos = p.positions[cur.b];
      cur.lo = p.window > 0 ? max(0, cur.pos - p.window + 1) : 0;
      cur.first_page = cur.lo / kPage;
      cur.trow = p.table + static_cast<long long>(cur.b) * p.pages_per_row;
    };
    int blk = 0, round = 0, ip = 0;  // ring block and its use, page of this consumer
    bool vnext = false;              // the page's V comes next
    bool done = lane >= kWarps;
    int page = 0;
    bool valid = false;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (lane 0's clock, here and below: the lanes give up in the same turn, as the votes need)
    uint64_t last_ns = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
    bool moved_since = false;
    for (uint32_t it = 1;; ++it) {
      bool moved = false;
      // (the lanes poll: none waits for another's consumer)
      if (!done && (round == 0 || mbar_test_wait(smem_addr(empty + blk), (round - 1) & 1))) {
        const uint32_t fb = smem_addr(full + blk);
        const uint32_t dst = smem_addr(smem + L::ring + size_t(w * kRing + blk) * L::kBlock);
        if (!vnext) {
          Page& pi = info[w * kPages + ip % kPages];
          if (gi >= re) {
            pi.flags = kEnd;
            mbar_arrive(fb);
            done = true;
          } else {
            page = entry;
            valid = page >= 0 && page < p.num_pages;
            const int lp = cur.first_page + cur.j;
            pi.b = cur.b;
            pi.h = cur.h;
            pi.klo = valid ? max(cur.lo - lp * kPage, 0) : 0;
            pi.khi = valid ? min(cur.pos - lp * kPage + 1, kPage) : 0;
            const bool first = gi == rb || cur.j == 0;
            pi.flags = (first ? kFirst : 0) | (gi + 1 == re ? kRunEnd : 0) |
                       (gi + 1 == re || cur.j + 1 == cur.np ? kLast : 0) |
                       (gi - cur.j >= rb && gi - cur.j + cur.np <= re ? kWhole : 0);
            if (!valid && p.status != nullptr) atomicOr(p.status, LNK_DEV_BAD_PAGE);
            if (first) {  // the piece's query rows, into L1
              const char* qsrc = reinterpret_cast<const char*>(
                  p.q + (static_cast<size_t>(cur.b) * p.hq + static_cast<size_t>(cur.h) * G) * D);
              for (int o = 0; o < G * D * 2; o += 128)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<uint64_t>(qsrc + o)));
            }
            if (valid) {
              mbar_arrive_expect_tx(fb, L::kBlock);
              bulk_load(dst, p.k_pool4 + (static_cast<size_t>(cur.h) * p.num_pages + page) * L::kBlock, L::kBlock, fb);
            } else {
              mbar_arrive(fb);
            }
            vnext = true;
          }
        } else {
          if (valid) {
            mbar_arrive_expect_tx(fb, L::kBlock);
            bulk_load(dst, p.v_pool4 + (static_cast<size_t>(cur.h) * p.num_pages + page) * L::kBlock, L::kBlock, fb);
          } else {
            mbar_arrive(fb);
          }
          vnext = false;
          ++ip;
          // this consumer's next page
          if (++gi < re) {
            if (++cur.j == cur.np) next_pair();
            entry = cur.trow[cur.first_page + cur.j];
          }
        }
        if (++blk == kRing) {
          blk = 0;
          ++round;
        }
        moved = true;
      }
      if (__all_sync(0xffffffffu, done)) break;
      moved = __any_sync(0xffffffffu, moved);
      moved_since = moved_since || moved;
      if (!moved) __nanosleep(32);
      // bounded: stop when nothing has moved for the waits' limit
      if ((it & 255u) == 0) {
        const uint64_t now = __shfl_sync(0xffffffffu, global_timer_ns(), 0);
        if (moved_since) last_ns = now;
        moved_since = false;
        if (__any_sync(0xffffffffu, *abort_flag != 0) || now - last_ns > 2 * kWaitLimitNs) {
          *abort_flag = 1;
          break;
        }
      }
    }
    // Drain: do not leave the CTA while a copy may still land in its memory.
    if (lane < kWarps) {
      for (int i = 0; i < kRing; ++i) {  // the last use of each block
        const int uses = round + (i < blk ? 1 : 0);
        if (uses == 0) continue;
        const uint64_t t1 = global_timer_ns();
        while (!mbar_try_wait(smem_addr(full + i), (uses - 1) & 1) && global_timer_ns() - t1 < kWaitLimitNs) {
        }
      }
    }
    if (*abort_flag && lane == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
    return;
  }

  // ============================== consumers ==============================
  const int c = lane & 3;
  const int r = lane >> 2;
  const int kperm = (r >> 1) + 4 * (r & 1);  // key within a group of 8
  // blocks of this lane's key dimensions, and of its value dimensions
  const int kb = (c * KW) / 2;
  const int vb = D == 128 ? r : r / 2;
  // where a piece's state lies: the run's first in its slot, the last in the ring
  auto piece_state = [&](int i) {
    return i & 1 ? reinterpret_cast<const float*>(smem + L::ring + size_t(i >> 1) * kRing * L::kBlock)
                 : state + size_t(i >> 1) * L::kStateFloats;
  };
  uint64_t* full = full_bar + warp * kRing;
  uint64_t* empty = empty_bar + warp * kRing;
  const uint8_t* ring = smem + L::ring + size_t(warp) * kRing * L::kBlock;
  uint32_t qf[KS][2];
  float o[KS][4];
  float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;  // heads 2c, 2c + 1
  int blk = 0, phase = 0;  // the next block of the ring, and its phase

  // four outputs of head g of pair q (pairs are in the order of the output's heads)
  auto store_out = [&](int q, int g, int d, const float4& acc, float sum) {
    const float inv = sum > 0.f ? p.out_scale / sum : 0.f;
    *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(q) * G + g) * D + d) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  };
  constexpr int kAll = kWarps * 32;
  constexpr int D4 = D / 4;

  // Two passes: the real one, and before it, while the previous kernel on the
  // stream still runs, a dry one of the final phase that touches no global memory.
  // It brings that phase's code into the instruction cache before the end, when every
  // warp waits for it.
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const bool dry = pass == 0;
    if (!dry) {
      // (the previous kernel writes q and the pools)
      asm volatile("griddepcontrol.wait;" ::: "memory");
      zero_rows();
    for (int ip = 0;; ++ip) {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(full + blk), phase, abort_flag))) break;
      const Page& pi = info[warp * kPages + ip % kPages];
      const int flags = pi.flags, klo = pi.klo, khi = pi.khi;
      if (flags & kEnd) break;
      if (flags & kFirst) {
        const uint16_t* qs = p.q + (static_cast<size_t>(pi.b) * p.hq + static_cast<size_t>(pi.h) * G + r) * D + c * (D / 4);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {  // dimensions c D/4 + 4 kk .. + 3 of head r
          const uint2 w = r < G ? *reinterpret_cast<const uint2*>(qs + 4 * kk) : make_uint2(0u, 0u);
          qf[kk][0] = bf16x2_to_f16x2(w.x);
          qf[kk][1] = bf16x2_to_f16x2(w.y);
        }
#pragma unroll
        for (int dt = 0; dt < KS; ++dt) o[dt][0] = o[dt][1] = o[dt][2] = o[dt][3] = 0.f;
        m_a = m_b = -INFINITY;
        l_a = l_b = 0.f;
      }
      const bool work = khi > klo;
      const bool partial = klo > 0 || khi < kPage;
      const uint8_t* kp = ring + blk * L::kBlock;
      const int kblk = blk;
      if (++blk == kRing) {
        blk = 0;
        phase ^= 1;
      }
      const uint8_t* vp = ring + blk * L::kBlock;
      uint32_t pb[4][2];  // P^T, keys in the order of the value pairs
      if (work) {
        // ---- S^T = K Q^T ----
        float sc[4][4];
#pragma unroll
        for (int t = 0; t < 4; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
        {
          // scales of keys kperm + 8 i, i = 0 .. 7, in pairs (i, i + 1), for the lane's blocks
          constexpr int NBLK = D == 64 ? 1 : 2;
          uint32_t ks[NBLK][4];
#pragma unroll
          for (int n = 0; n < NBLK; ++n) {
            const uint4 w = *reinterpret_cast<const uint4*>(kp + 32 * D + ((r >> 1) * KS + kb + n) * 16);
            const uint32_t sel = (r & 1) ? 0x7531u : 0x6420u;
            e4m3x4_to_f16x2x2(__byte_perm(w.x, w.y, sel), ks[n][0], ks[n][1]);
            e4m3x4_to_f16x2x2(__byte_perm(w.z, w.w, sel), ks[n][2], ks[n][3]);
          }
          uint32_t kw[8][KW];  // code words of keys kperm + 8 i
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint8_t* src = kp + (kperm + 8 * i) * (D / 2) + c * (KW * 4);
            if constexpr (D == 128) {
              const uint4 w = *reinterpret_cast<const uint4*>(src);
              kw[i][0] = w.x; kw[i][1] = w.y; kw[i][2] = w.z; kw[i][3] = w.w;
            } else if constexpr (D == 64) {
              const uint2 w = *reinterpret_cast<const uint2*>(src);
              kw[i][0] = w.x; kw[i][1] = w.y;
            } else {
#pragma unroll
              for (int x = 0; x < KW; ++x) kw[i][x] = reinterpret_cast<const uint32_t*>(src)[x];
            }
          }
          // the keys are in registers: their block may be loaded again
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(empty + kblk));
#pragma unroll
          for (int x = 0; x < KW; ++x) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              // word x lies in the lane's first or second block
              uint32_t sp;
              if constexpr (D == 64) sp = ks[0][t];
              else if constexpr (D == 128) sp = ks[x >> 1][t];
              else sp = x == 0 ? ks[0][t] : (x == 2 ? ks[1][t] : ((c & 1) ? ks[1][t] : ks[0][t]));
              uint32_t ra[4], rb[4];  // rows r (key 2t) and r + 8 (key 2t + 1), two k-steps each
              e2m1x8_to_f16x2x4(kw[2 * t][x], ra);
              e2m1x8_to_f16x2x4(kw[2 * t + 1][x], rb);
              const uint32_t sa = low2(sp), sb = high2(sp);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                ra[i] = mul_f16x2(ra[i], sa);
                rb[i] = mul_f16x2(rb[i], sb);
              }
              mma_f16_16816(sc[t], ra[0], rb[0], ra[1], rb[1], qf[2 * x][0], qf[2 * x][1]);
              mma_f16_16816(sc[t], ra[2], rb[2], ra[3], rb[3], qf[2 * x + 1][0], qf[2 * x + 1][1]);
            }
          }
        }
        // ---- mask, online softmax (log2 domain) ----
        float mx_a = -INFINITY, mx_b = -INFINITY;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (partial) {
              const int key = 16 * t + 8 * (i >> 1) + kperm;
              if (key < klo || key >= khi) sc[t][i] = -INFINITY;
            }
          }
          mx_a = fmax3(mx_a, sc[t][0], sc[t][2]);
          mx_b = fmax3(mx_b, sc[t][1], sc[t][3]);
        }
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
          mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
        }
        // (the scale is positive: the largest product is the largest score's)
        const float mn_a = fmaxf(m_a, fmaf(mx_a, p.scale_log2, -kHeadroomLog2));
        const float mn_b = fmaxf(m_b, fmaf(mx_b, p.scale_log2, -kHeadroomLog2));
        const bool same_max = __all_sync(0xffffffffu, mn_a == m_a && mn_b == m_b);
        const float base_a = mn_a == -INFINITY ? 0.f : mn_a;
        const float base_b = mn_b == -INFINITY ? 0.f : mn_b;
        if (!same_max) {  // a running max moved: O and the sums follow
          const float al_a = ex2_approx(m_a - base_a), al_b = ex2_approx(m_b - base_b);
          l_a *= al_a;
          l_b *= al_b;
#pragma unroll
          for (int dt = 0; dt < KS; ++dt) {
            o[dt][0] *= al_a;
            o[dt][1] *= al_b;
            o[dt][2] *= al_a;
            o[dt][3] *= al_b;
          }
        }
        m_a = mn_a;
        m_b = mn_b;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float p0 = ex2_approx(fmaf(sc[t][0], p.scale_log2, -base_a));
          const float p1 = ex2_approx(fmaf(sc[t][1], p.scale_log2, -base_b));
          const float p2 = ex2_approx(fmaf(sc[t][2], p.scale_log2, -base_a));
          const float p3 = ex2_approx(fmaf(sc[t][3], p.scale_log2, -base_b));
          l_a += p0 + p2;
          l_b += p1 + p3;
          pb[t][0] = movmatrix_trans(pack_f16x2(p0, p1));
          pb[t][1] = movmatrix_trans(pack_f16x2(p2, p3));
        }
      }
      if (!work) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(empty + kblk));
      }
      if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(full + blk), phase, abort_flag))) break;
      if (work) {
        // ---- O^T += V^T P^T ----
        // scales of keys c + 4 i in pairs (i, i + 1), for the lane's blocks; zero where masked
        constexpr int NVB = D == 96 ? 2 : 1;
        uint32_t vs[NVB][8];
#pragma unroll
        for (int n = 0; n < NVB; ++n) {
          const int b = n == 0 ? vb : 4 + r / 4;
          uint4 w = *reinterpret_cast<const uint4*>(vp + 32 * D + (c * KS + b) * 16);
          if (partial) {
            uint32_t* ww = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int key = c + 4 * i;
              if (key < klo || key >= khi) ww[i >> 2] &= ~(0xFFu << (8 * (i & 3)));
            }
          }
          e4m3x4_to_f16x2x2(w.x, vs[n][0], vs[n][1]);
          e4m3x4_to_f16x2x2(w.y, vs[n][2], vs[n][3]);
          e4m3x4_to_f16x2x2(w.z, vs[n][4], vs[n][5]);
          e4m3x4_to_f16x2x2(w.w, vs[n][6], vs[n][7]);
        }
        constexpr int VW = D == 128 ? 2 : 1;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          uint32_t vw[4][VW];
          uint32_t vh[4];  // D = 96: dimensions 64 + 4 r .. + 3
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint8_t* src = vp + (c + 4 * (4 * t + i)) * (D / 2);
            if constexpr (D == 128) {
              const uint2 w = *reinterpret_cast<const uint2*>(src + 8 * r);
              vw[i][0] = w.x;
              vw[i][1] = w.y;
            } else {
              vw[i][0] = *reinterpret_cast<const uint32_t*>(src + 4 * r);
              if constexpr (D == 96) vh[i] = *reinterpret_cast<const uint16_t*>(src + 32 + 2 * r);
            }
          }
#pragma unroll
          for (int y = 0; y < VW; ++y) {
            uint32_t e0[4], o0[4], e1[4], o1[4];
            e2m1x8_to_f16x2x4(mix_even(vw[0][y], vw[1][y]), e0);
            e2m1x8_to_f16x2x4(mix_odd(vw[0][y], vw[1][y]), o0);
            e2m1x8_to_f16x2x4(mix_even(vw[2][y], vw[3][y]), e1);
            e2m1x8_to_f16x2x4(mix_odd(vw[2][y], vw[3][y]), o1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mma_f16_16816(o[4 * y + i], mul_f16x2(e0[i], vs[0][2 * t]), mul_f16x2(o0[i], vs[0][2 * t]),
                            mul_f16x2(e1[i], vs[0][2 * t + 1]), mul_f16x2(o1[i], vs[0][2 * t + 1]), pb[t][0], pb[t][1]);
          }
          if constexpr (D == 96) {
            // the 16-bit words of two keys, side by side, convert as one word each
            uint32_t e0[4], e1[4];
            e2m1x8_to_f16x2x4(mix_even(vh[0], vh[1]) | (mix_odd(vh[0], vh[1]) << 16), e0);
            e2m1x8_to_f16x2x4(mix_even(vh[2], vh[3]) | (mix_odd(vh[2], vh[3]) << 16), e1);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mma_f16_16816(o[4 + i], mul_f16x2(e0[i], vs[NVB - 1][2 * t]), mul_f16x2(e0[2 + i], vs[NVB - 1][2 * t]),
                            mul_f16x2(e1[i], vs[NVB - 1][2 * t + 1]), mul_f16x2(e1[2 + i], vs[NVB - 1][2 * t + 1]),
                            pb[t][0], pb[t][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(empty + blk));
      if (++blk == kRing) {
        blk = 0;
        phase ^= 1;
      }
      if (!(flags & kLast)) continue;

      float la = l_a, lb = l_b;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        la += __shfl_xor_sync(0xffffffffu, la, off);
        lb += __shfl_xor_sync(0xffffffffu, lb, off);
      }
      const int ob = pi.b, oh = pi.h;
      if (flags & kWhole) {
        // ---- a whole pair: this lane's dimensions of heads 2c and 2c + 1 ----
        const float ia = la > 0.f ? p.out_scale / la : 0.f, ib = lb > 0.f ? p.out_scale / lb : 0.f;
        uint16_t* oa = p.out + (static_cast<size_t>(ob) * p.hq + static_cast<size_t>(oh) * G + 2 * c) * D;
#pragma unroll
        for (int dt = 0; dt < KS; dt += 2) {
          const int d = D == 128 ? 16 * r + 2 * dt : (dt < 4 ? 8 * r + 2 * dt : 64 + 4 * r);
          if (2 * c < G)
            *reinterpret_cast<uint2*>(oa + d) = make_uint2(pack_bf16x2(o[dt][0] * ia, o[dt][2] * ia),
                                                           pack_bf16x2(o[dt + 1][0] * ia, o[dt + 1][2] * ia));
          if (2 * c + 1 < G)
            *reinterpret_cast<uint2*>(oa + D + d) = make_uint2(pack_bf16x2(o[dt][1] * ib, o[dt][3] * ib),
                                                               pack_bf16x2(o[dt + 1][1] * ib, o[dt + 1][3] * ib));
        }
        continue;
      }
      // ---- a piece of a longer pair: its state into shared memory ----
      const int piece = 2 * warp + (flags & kRunEnd ? 1 : 0);
      if (lane < 4) {
        smax[piece * kMaxGroup + 2 * c] = m_a;
        smax[piece * kMaxGroup + 2 * c + 1] = m_b;
        ssum[piece * kMaxGroup + 2 * c] = la;
        ssum[piece * kMaxGroup + 2 * c + 1] = lb;
      }
      if (lane == 0) piece_pair[piece] = ob * p.hkv + oh;
      float* oa = const_cast<float*>(piece_state(piece)) + (2 * c) * L::kOStride;
#pragma unroll
      for (int dt = 0; dt < KS; dt += 2) {
        // d-tiles dt, dt + 1: four consecutive dimensions
        const int d = D == 128 ? 16 * r + 2 * dt : (dt < 4 ? 8 * r + 2 * dt : 64 + 4 * r);
        *reinterpret_cast<float4*>(oa + d) = make_float4(o[dt][0], o[dt][2], o[dt + 1][0], o[dt + 1][2]);
        *reinterpret_cast<float4*>(oa + L::kOStride + d) = make_float4(o[dt][1], o[dt][3], o[dt + 1][1], o[dt + 1][3]);
      }
    }
    }

    // ================= all runs are done: merge the pieces ==================
    // (every consumer warp comes here, whatever ended its loop)
    named_barrier_sync(1, kAll);
    // Pieces of one pair are neighbours.  Bit i: piece i is there / begins a pair.
    const int mine = dry ? (lane == 0 ? 0 : -1) : (lane < kPieces ? piece_pair[lane] : -1);
    const unsigned there = __ballot_sync(0xffffffffu, mine >= 0);
    const unsigned before = there & ((1u << lane) - 1u);
    const int prev = __shfl_sync(0xffffffffu, mine, before ? 31 - __clz(before) : 0);
    const unsigned heads = __ballot_sync(0xffffffffu, mine >= 0 && (before == 0u || prev != mine));
    const int items = G * D4;  // of a pair: four dimensions of a head each
    const int total_items = __popc(heads) * items;
    const bool cut0 = dry || shared[2] != 0, cut1 = !dry && shared[5] != 0;
    for (int idx = tid; idx < total_items; idx += kAll) {
      const int gidx = idx / items, it = idx - gidx * items;
      const int g = it / D4, d = (it % D4) * 4;
      unsigned rest = heads;
      for (int i = 0; i < gidx; ++i) rest &= rest - 1;
      const int at = __ffs(rest) - 1;
      rest &= rest - 1;
      const unsigned mask = there & (rest ? (1u << (__ffs(rest) - 1)) - (1u << at) : ~0u << at);
      const int q = dry ? 0 : piece_pair[at];
      float M = -INFINITY;
      for (unsigned m = mask; m; m &= m - 1) M = fmaxf(M, smax[(__ffs(m) - 1) * kMaxGroup + g]);
      const float base = M == -INFINITY ? 0.f : M;  // (then every weight is 2^-inf = 0)
      float Ls = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (unsigned m = mask; m; m &= m - 1) {
        const int i = __ffs(m) - 1;
        const float f = ex2_approx(smax[i * kMaxGroup + g] - base);
        const float4 v = *reinterpret_cast<const float4*>(piece_state(i) + g * L::kOStride + d);
        Ls += ssum[i * kMaxGroup + g] * f;
        acc.x += v.x * f;
        acc.y += v.y * f;
        acc.z += v.z * f;
        acc.w += v.w * f;
      }
      if (dry) continue;
      if ((cut0 && q == shared[0]) || (cut1 && q == shared[3])) {  // the partial's place in the workspace: pair + chunk
        const size_t row = (static_cast<size_t>(q) + chunk) * G + g;
        *reinterpret_cast<float4*>(p.ws_o + row * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(p.ws_ml + row * 2) = make_float2(M, Ls);
      } else {
        store_out(q, g, d, acc, Ls);
      }
    }
    if (!cut0 && !cut1) continue;
    // ---- pairs shared with other CTAs: count the pair's finished chunks; the
    // last CTA merges them (the barrier and the fence publish the partials) ----
    named_barrier_sync(1, kAll);
    if (tid < 2) {
      int last = dry;
      if (!dry && shared[tid * 3 + 2] != 0) {
        const int q = shared[tid * 3];
        __threadfence();
        last = atomicAdd(p.ws_count + q, 1) == shared[tid * 3 + 2] - 1;
        __threadfence();
        if (last) p.ws_count[q] = 0;  // ready for the next call
      }
      arrived_last[tid] = last;
    }
    named_barrier_sync(1, kAll);
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      if (!arrived_last[which]) continue;
      const int q = dry ? 0 : shared[which * 3], nseg = dry ? 1 : shared[which * 3 + 2];
      const size_t seg0 = dry ? 0 : static_cast<size_t>(q) + shared[which * 3 + 1];
      for (int it = tid; it < items; it += kAll) {
        const int g = it / D4, d = (it % D4) * 4;
        float M = -INFINITY, Ls = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kAtOnce = 4;
#pragma unroll 1
        for (int s0 = 0; s0 < nseg; s0 += kAtOnce) {  // partials in their order, several loads in flight
          float2 ml[kAtOnce];
          float4 v[kAtOnce];
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) {
            const size_t row = (seg0 + min(s0 + u, nseg - 1)) * G + g;
            ml[u] = make_float2(-INFINITY, 0.f);
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!dry) {  // (the previous kernel may still write the workspace then)
              ml[u] = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + row);
              v[u] = __ldcg(reinterpret_cast<const float4*>(p.ws_o + row * D + d));
            }
            if (s0 + u >= nseg) ml[u].x = -INFINITY;
          }
          float mn = M;
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) mn = fmaxf(mn, ml[u].x);
          const float base = mn == -INFINITY ? 0.f : mn;
          const float f0 = ex2_approx(M - base);
          Ls *= f0;
          acc.x *= f0;
          acc.y *= f0;
          acc.z *= f0;
          acc.w *= f0;
#pragma unroll
          for (int u = 0; u < kAtOnce; ++u) {
            const float f = ex2_approx(ml[u].x - base);
            Ls += ml[u].y * f;
            acc.x += v[u].x * f;
            acc.y += v[u].y * f;
            acc.z += v[u].z * f;
            acc.w += v[u].w * f;
          }
          M = mn;
        }
        if (!dry) store_out(q, g, d, acc, Ls);
      }
    }
  }
  if (*abort_flag && lane == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
}

template <int D>
cudaError_t launch_t(const DecodeParams& p, const DecodeLaunch& launch, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(launch.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = launch.smem_bytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode4_kernel<D>, p);
}

template <int D>
cudaError_t prepare_t(int B, DecodeLaunch* launch) {
  const size_t bytes = Smem<D>::bytes(B);
  const void* fn = reinterpret_cast<const void*>(decode4_kernel<D>);
  cudaError_t err = set_max_dynamic_smem(fn, static_cast<int>(bytes));
  if (err != cudaSuccess) return err;
  launch->smem_bytes = static_cast<int>(bytes);
  launch->grid = device_sm_count();
  launch->mode = 0;
  return cudaSuccess;
}

}  // namespace

cudaError_t decode4_prepare(int head_dim, int B, DecodeLaunch* launch) {
  switch (head_dim) {
    case 64: return prepare_t<64>(B, launch);
    case 96: return prepare_t<96>(B, launch);
    case 128: return prepare_t<128>(B, launch);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_decode4(const DecodeParams& p, int head_dim, const DecodeLaunch& launch, cudaStream_t stream) {
  if (p.B == 0) return cudaSuccess;
  switch (head_dim) {
    case 64: return launch_t<64>(p, launch, stream);
    case 96: return launch_t<96>(p, launch, stream);
    case 128: return launch_t<128>(p, launch, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
