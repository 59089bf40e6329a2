// Paged split-KV decode attention over 4-bit pools (LNK_KV_E2M1).
//
// The work decomposition, the partial results of cut pairs and their merge are
// decode.cu's (decode_plan.cuh).  What differs is the CTA's inside, because a
// page of one head is only 36 D bytes of K and of V: at the rate HBM delivers
// them, an SM has about 390 cycles for the 16384 elements of a page's K and V
// (D = 128), so the instructions spent per page decide, and everything that is
// paid per page and warp is paid by ONE warp per page:
//  * warps 0 .. kWarps - 1, consumers: warp w takes whole pages (64 keys), those
//    with index w modulo kWarps in the CTA's stream, with an online softmax of
//    its own; one set of maxima, votes and barriers serves 64 keys;
//  * producer warp: one lane walks the CTA's page-heads and loads each page's K
//    and V (two contiguous blocks of 36 D bytes, 1-D bulk copies) into a ring of
//    stages; a segment's query rows go with the first page that each warp
//    gets of it;
//  * epilogue warp: merges the states of the warps that had pages of a segment
//    (at most min(kWarps, pages) of them) and writes the output or the partial.
//
// Arithmetic.  A code times its block's E4M3 scale has at most five significant
// bits and lies in f16's range (2^-10 .. 2688), so the converted keys and values
// are exact; the query is rounded to f16 (exact in the range the header states),
// the probabilities to f16 (relative 2^-11, on values that sum to the
// denominator kept in float32), and all sums are float32.
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

constexpr int kWarps = 4;  // consumer warps
constexpr int kProducerWarp = kWarps;
constexpr int kEpilogueWarp = kWarps + 1;
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kCtasPerSm = 2;
// K + V pages in the ring.  A multiple of the warps: page k goes to stage
// k % kStages and warp k % kWarps, so that every stage belongs to one warp.  (A
// stage shared by two warps would be waited on by parity from two places: a warp
// that is ahead could take the phase before the last for the one it waits for.)
constexpr int kStages = 8;
static_assert(kStages % kWarps == 0, "a stage's phases are waited for by one warp, in order");
constexpr int kPairWhole = 1;
constexpr int kEnd = 2;
constexpr int kFirst = 4;   // the warp's first page of the segment (the stage has its query rows)
constexpr int kLast = 8;    // the warp's last page of the segment

struct Stage {
  int b, h, klo, khi, flags, seg, nseg, c0, pages;  // pages: of the segment, in this chunk
};

template <int D>
struct Smem {
  static constexpr int kSlots = D == 128 ? 1 : 2;     // hand-off slots per consumer warp (what fits)
  static constexpr int kPageBytes = 36 * D;
  static constexpr int kStageBytes = 2 * kPageBytes;  // K, then V
  static constexpr int kQBytes = kMaxGroup * D * 2;
  static constexpr int kOStride = D + 4;              // padded staging row
  static constexpr int kSlotFloats = kMaxGroup * kOStride;
  static constexpr size_t stages = 0;
  static constexpr size_t qbuf = stages + size_t(kStages) * kStageBytes;
  static constexpr size_t ostage = qbuf + size_t(kStages) * kQBytes;          // [kWarps][kSlots][kMaxGroup][kOStride]
  static constexpr size_t mstage = ostage + size_t(kWarps) * kSlots * kSlotFloats * 4;  // [kWarps][kSlots][kMaxGroup]
  static constexpr size_t lstage = mstage + size_t(kWarps) * kSlots * kMaxGroup * 4;
  static constexpr size_t epi = lstage + size_t(kWarps) * kSlots * kMaxGroup * 4;  // [2][kMaxGroup]: max, sum
  // full[kStages], empty[kStages], slot_full[kWarps][kSlots], slot_empty[kWarps][kSlots]
  static constexpr size_t bars = epi + 2 * kMaxGroup * 4;
  static constexpr size_t info = bars + (2 * kStages + 2 * kWarps * kSlots) * sizeof(uint64_t);
  static constexpr size_t slot_info = info + kStages * sizeof(Stage);
  static constexpr size_t misc = slot_info + kWarps * kSlots * sizeof(Stage);  // abort, longest pair, warp sums
  static constexpr size_t pref = misc + (2 + kWarps + 2) * 4;
  static_assert(kStageBytes % 128 == 0 && kQBytes % 16 == 0 && bars % 8 == 0, "copies land on 16-byte boundaries");
  static size_t bytes(int B) { return pref + size_t(B + 1) * 4 + 128; }  // + alignment slack
};

__device__ __forceinline__ uint32_t low2(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t h) { return __byte_perm(h, h, 0x3232); }

// Byte order of eight codes of two keys, one dimension of both per byte: the
// even dimensions' codes (low four bits of a and of b) ...
__device__ __forceinline__ uint32_t mix_even(uint32_t a, uint32_t b) {
  return (a & 0x0F0F0F0Fu) | ((b << 4) & 0xF0F0F0F0u);
}
// ... and the odd ones'.
__device__ __forceinline__ uint32_t mix_odd(uint32_t a, uint32_t b) {
  return ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
}

template <int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) decode4_kernel(const DecodeParams p) {
  using L = Smem<D>;
  constexpr int kSlots = L::kSlots;
  constexpr int KS = D / 16;  // k-steps of Q.K, d-tiles of P.V, blocks of a row
  constexpr int KW = D / 32;  // words of a key row per lane
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + L::bars);
  uint64_t* empty_bar = full_bar + kStages;
  uint64_t* slot_full = empty_bar + kStages;           // [kWarps][kSlots]
  uint64_t* slot_empty = slot_full + kWarps * kSlots;  // [kWarps][kSlots]
  Stage* info = reinterpret_cast<Stage*>(smem + L::info);
  Stage* slot_info = reinterpret_cast<Stage*>(smem + L::slot_info);
  float* ost = reinterpret_cast<float*>(smem + L::ostage);
  float* mst = reinterpret_cast<float*>(smem + L::mstage);
  float* lst = reinterpret_cast<float*>(smem + L::lstage);
  int* misc = reinterpret_cast<int*>(smem + L::misc);  // [0] abort, [1] longest pair, [2..] warp sums of the scan
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

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_addr(full_bar + s), 1);
      mbar_init(smem_addr(empty_bar + s), 1);
    }
    for (int i = 0; i < kWarps * kSlots; ++i) {
      mbar_init(smem_addr(slot_full + i), 1);
      mbar_init(smem_addr(slot_empty + i), 1);
    }
    misc[0] = 0;
    misc[1] = 0;
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

  // Wait for the previous kernel on the stream (it writes q and the pools).
  // The producer waits later, right before its first copy.
  if (warp != kProducerWarp) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // rows with nothing to attend to get a zero output
    const int zt = warp < kProducerWarp ? tid : tid - 32;
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      if (pref[b + 1] == pref[b]) {
        uint32_t* o = reinterpret_cast<uint32_t*>(p.out + static_cast<size_t>(b) * p.hq * D);
        for (int i = zt; i < p.hq * D / 2; i += kThreads - 32) o[i] = 0u;
      }
    }
  }
  if (chunk >= nchunks) return;

  if (warp == kProducerWarp) {
    // ============================== producer ==============================
    if (lane != 0) return;
    long long start, end;
    if (pair_chunks) {
      const int b = static_cast<int>(chunk / p.hkv), h = static_cast<int>(chunk % p.hkv);
      const int np = pref[b + 1] - pref[b];
      start = static_cast<long long>(pref[b]) * p.hkv + static_cast<long long>(h) * np;
      end = start + np;
    } else {
      start = chunk * per;
      end = min(total, start + per);
    }
    int k = 0;
    bool stop = false, waited = false;
    if (start < end) {
      // ranges in order: the segment shared with the next chunk first, so that
      // cut pairs finish early
      Cursor cur;
      locate(cur, end - 1, pref, p, start, end, per, chunk);
      const long long last_seg = max(start, end - 1 - cur.j);
      const bool last_cut = (end - 1 - cur.j) + cur.np > end;
      const bool two = last_cut && last_seg > start;
      for (int rg = 0; rg < (two ? 2 : 1) && !stop; ++rg) {
        const long long rb = two && rg == 0 ? last_seg : start, re = two && rg == 1 ? last_seg : end;
        locate(cur, rb, pref, p, start, end, per, chunk);
        int seg_pages = 0, idx = 0;  // pages of the cursor's segment, and its page in it
        for (long long gi = rb; gi < re; ++gi, ++k) {
          if (gi == rb || cur.j == 0) {
            seg_pages = static_cast<int>(min(static_cast<long long>(cur.np - cur.j), re - gi));
            idx = 0;
          }
          const int lp = cur.first_page + cur.j;
          const int page = cur.trow[lp];
          const int s = k % kStages;
          if (k >= kStages && !mbar_wait(smem_addr(empty_bar + s), ((k / kStages) - 1) & 1, abort_flag)) {
            stop = true;
            break;
          }
          const bool first = idx < kWarps;
          const bool valid = page >= 0 && page < p.num_pages;
          Stage si;
          si.b = cur.b;
          si.h = cur.h;
          si.klo = max(cur.lo - lp * kPage, 0);
          si.khi = min(cur.pos - lp * kPage + 1, kPage);
          si.flags = (first ? kFirst : 0) | (seg_pages - 1 - idx < kWarps ? kLast : 0) | (cur.whole ? kPairWhole : 0);
          si.seg = cur.seg;
          si.nseg = cur.nseg;
          si.c0 = cur.c0;
          si.pages = seg_pages;
          if (!valid) {
            if (p.status != nullptr) atomicOr(p.status, LNK_DEV_BAD_PAGE);
            si.klo = si.khi = 0;
          }
          info[s] = si;
          const uint32_t fb = smem_addr(full_bar + s);
          const uint32_t q_bytes = first ? static_cast<uint32_t>(G * D * 2) : 0u;
          const uint32_t tx = (valid ? static_cast<uint32_t>(L::kStageBytes) : 0u) + q_bytes;
          if (tx) mbar_arrive_expect_tx(fb, tx); else mbar_arrive(fb);
          if (!waited) {  // (the previous kernel writes q and the pools)
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
          }
          if (q_bytes > 0) {
            const uint16_t* qsrc = p.q + (static_cast<size_t>(cur.b) * p.hq + static_cast<size_t>(cur.h) * G) * D;
            bulk_load(smem_addr(smem + L::qbuf + size_t(s) * L::kQBytes), qsrc, q_bytes, fb);
          }
          if (valid) {
            const uint32_t dst = smem_addr(smem + L::stages + size_t(s) * L::kStageBytes);
            const size_t at = (static_cast<size_t>(cur.h) * p.num_pages + page) * L::kPageBytes;
            bulk_load(dst, p.k_pool4 + at, L::kPageBytes, fb);
            bulk_load(dst + L::kPageBytes, p.v_pool4 + at, L::kPageBytes, fb);
          }
          ++idx;
          if (++cur.j == cur.np && gi + 1 < re) locate(cur, gi + 1, pref, p, start, end, per, chunk);
        }
      }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    // the end of the work: a stage without data for every consumer warp
    for (int w = 0; w < kWarps && !stop; ++w, ++k) {
      const int s = k % kStages;
      if (k >= kStages && !mbar_wait(smem_addr(empty_bar + s), ((k / kStages) - 1) & 1, abort_flag)) {
        stop = true;  // the consumers stop on the abort flag
        break;
      }
      Stage si{};
      si.flags = kEnd;
      info[s] = si;
      mbar_arrive(smem_addr(full_bar + s));
    }
    // Drain: do not leave the CTA while a copy may still land in its memory.
    for (int kk = max(0, k - kStages); kk < k; ++kk) {
      const uint32_t fb = smem_addr(full_bar + kk % kStages);
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(fb, (kk / kStages) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {
      }
    }
    if (*abort_flag && p.status != nullptr) atomicOr(p.status, LNK_DEV_TIMEOUT);
    return;
  }

  if (warp == kEpilogueWarp) {
    // ============================== epilogue ==============================
    float* eml = reinterpret_cast<float*>(smem + L::epi);  // [2][kMaxGroup]: max, sum per head
    constexpr int D4 = D / 4;
    int seq = 0;    // lane w: segments taken from consumer warp w
    int first = 0;  // consumer warp with the next segment's first page
    for (;;) {
      const int n0 = __shfl_sync(0xffffffffu, seq, first);
      if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(slot_full + first * kSlots + n0 % kSlots), (n0 / kSlots) & 1,
                                             abort_flag)))
        break;
      const Stage si = slot_info[first * kSlots + n0 % kSlots];
      if (si.flags & kEnd) break;
      const int nw = min(kWarps, si.pages);  // warps with pages of the segment: first, first + 1, ...
      bool ok = true;
      int slot_of[kWarps];  // their hand-off slots
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const int w = (first + i) % kWarps;
        const int n = __shfl_sync(0xffffffffu, seq, w);
        slot_of[i] = w * kSlots + n % kSlots;
        if (i > 0 && i < nw)
          ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_addr(slot_full + slot_of[i]), (n / kSlots) & 1, abort_flag));
      }
      if (!ok) break;
      const bool whole = (si.flags & kPairWhole) != 0;
      uint16_t* out_pair = p.out + (static_cast<size_t>(si.b) * p.hq + static_cast<size_t>(si.h) * G) * D;
      const int q = si.b * p.hkv + si.h;
      // per head: merged max and sum of the warps
      if (lane < G) {
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; ++i)
          if (i < nw) M = fmaxf(M, mst[slot_of[i] * kMaxGroup + lane]);
        float Ls = 0.f;
        if (M != -INFINITY) {
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            if (i >= nw) continue;
            const float mw = mst[slot_of[i] * kMaxGroup + lane];
            if (mw != -INFINITY) Ls += lst[slot_of[i] * kMaxGroup + lane] * exp2f(mw - M);
          }
        }
        eml[lane] = M;
        eml[kMaxGroup + lane] = Ls;
      }
      __syncwarp();
      for (int it = lane; it < G * D4; it += 32) {
        const int g = it / D4, d = (it % D4) * 4;
        const float M = eml[g], Ls = eml[kMaxGroup + g];
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (M != -INFINITY) {
#pragma unroll
          for (int i = 0; i < kWarps; ++i) {
            if (i >= nw) continue;
            const float mw = mst[slot_of[i] * kMaxGroup + g];
            const float f = mw == -INFINITY ? 0.f : exp2f(mw - M);
            const float4 v = *reinterpret_cast<const float4*>(ost + size_t(slot_of[i]) * L::kSlotFloats + g * L::kOStride + d);
            acc.x += v.x * f;
            acc.y += v.y * f;
            acc.z += v.z * f;
            acc.w += v.w * f;
          }
        }
        if (whole) {
          const float inv = Ls > 0.f ? p.out_scale / Ls : 0.f;
          uint2 pk;
          pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
          pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(out_pair + g * D + d) = pk;
        } else {
          *reinterpret_cast<float4*>(p.ws_o + (static_cast<size_t>(si.seg) * G + g) * D + d) = acc;
          if (d == 0) {
            p.ws_ml[(static_cast<size_t>(si.seg) * G + g) * 2 + 0] = M;
            p.ws_ml[(static_cast<size_t>(si.seg) * G + g) * 2 + 1] = Ls;
          }
        }
      }
      __syncwarp();
      // the warps' slots are consumed
      {
        const int i = (lane - first + kWarps) % kWarps;
        if (lane < kWarps && i < nw) {
          mbar_arrive(smem_addr(slot_empty + lane * kSlots + seq % kSlots));
          ++seq;
        }
      }
      first = (first + si.pages) % kWarps;
      if (!whole) {
        // publish the partial, then count the pair's finished segments
        __threadfence();
        __syncwarp();
        int last = 0;
        if (lane == 0) {
          const int old = atomicAdd(p.ws_count + q, 1);
          last = old == si.nseg - 1;
          if (last) p.ws_count[q] = 0;  // ready for the next call
        }
        last = __shfl_sync(0xffffffffu, last, 0);
        if (last) {
          __threadfence();
          const size_t seg0 = static_cast<size_t>(q + si.c0);
          const int nsg = si.nseg;
          // pass 1: per head, online max and sum over the pair's segments; lane
          // handles head lane % G of segments lane / G, lane / G + 32 / G, ...
          float rm = -INFINITY, rl = 0.f;
          for (int i = lane; i < nsg * G; i += 32) {
            const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.ws_ml) + seg0 * G + i);
            if (ml.x != -INFINITY) {
              const float mn = fmaxf(rm, ml.x);
              rl = rl * exp2f(rm - mn) + ml.y * exp2f(ml.x - mn);
              rm = mn;
            }
          }
          for (int off = G; off < 32; off <<= 1) {
            const float om = __shfl_xor_sync(0xffffffffu, rm, off);
            const float ol = __shfl_xor_sync(0xffffffffu, rl, off);
            const float mn = fmaxf(rm, om);
            if (mn != -INFINITY) {
              rl = (rm == -INFINITY ? 0.f : rl * exp2f(rm - mn)) + (om == -INFINITY ? 0.f : ol * exp2f(om - mn));
              rm = mn;
            }
          }
          __syncwarp();
          if (lane < G) {
            eml[lane] = rm;
            eml[kMaxGroup + lane] = rl;
          }
          __syncwarp();
          // pass 2: weighted sum of the partial outputs (independent loads)
          for (int it = lane; it < G * D4; it += 32) {
            const int g = it / D4, d = (it % D4) * 4;
            const float M = eml[g], Ls = eml[kMaxGroup + g];
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            if (M != -INFINITY) {
              for (int sg = 0; sg < nsg; ++sg) {
                const size_t row = (seg0 + sg) * G + g;
                const float mseg = __ldcg(p.ws_ml + row * 2);
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p.ws_o + row * D + d));
                const float f = mseg == -INFINITY ? 0.f : exp2f(mseg - M);
                acc.x += v.x * f;
                acc.y += v.y * f;
                acc.z += v.z * f;
                acc.w += v.w * f;
              }
            }
            const float inv = Ls > 0.f ? p.out_scale / Ls : 0.f;
            uint2 pk;
            pk.x = pack_bf16x2(acc.x * inv, acc.y * inv);
            pk.y = pack_bf16x2(acc.z * inv, acc.w * inv);
            *reinterpret_cast<uint2*>(out_pair + g * D + d) = pk;
          }
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
  uint32_t qf[KS][2];
  float o[KS][4];
  float m_a = -INFINITY, m_b = -INFINITY, l_a = 0.f, l_b = 0.f;  // heads 2c, 2c + 1
  int nslot = 0;

  for (int k = warp;; k += kWarps) {
    const int s = k % kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(full_bar + s), (k / kStages) & 1, abort_flag))) break;
    const Stage si = info[s];
    const int slot = warp * kSlots + nslot % kSlots;
    if (si.flags & kEnd) {  // pass the end on to the epilogue
      if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(slot_empty + slot), ((nslot / kSlots) & 1) ^ 1, abort_flag))) break;
      if (lane == 0) {
        slot_info[slot] = si;
        mbar_arrive(smem_addr(slot_full + slot));
      }
      break;
    }
    if (si.flags & kFirst) {
      const uint16_t* qs = reinterpret_cast<const uint16_t*>(smem + L::qbuf + size_t(s) * L::kQBytes) + r * D + c * (D / 4);
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
    const bool work = si.khi > si.klo;
    if (work) {
      const uint8_t* kp = smem + L::stages + size_t(s) * L::kStageBytes;
      const uint8_t* vp = kp + L::kPageBytes;
      const bool partial = si.klo > 0 || si.khi < kPage;
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
          sc[t][i] *= p.scale_log2;
          if (partial) {
            const int key = 16 * t + 8 * (i >> 1) + kperm;
            if (key < si.klo || key >= si.khi) sc[t][i] = -INFINITY;
          }
        }
        mx_a = fmaxf(mx_a, fmaxf(sc[t][0], sc[t][2]));
        mx_b = fmaxf(mx_b, fmaxf(sc[t][1], sc[t][3]));
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, off));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, off));
      }
      const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
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
      uint32_t pb[4][2];  // P^T, keys in the order of the value pairs
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float p0 = ex2_approx(sc[t][0] - base_a), p1 = ex2_approx(sc[t][1] - base_b);
        const float p2 = ex2_approx(sc[t][2] - base_a), p3 = ex2_approx(sc[t][3] - base_b);
        l_a += p0 + p2;
        l_b += p1 + p3;
        pb[t][0] = movmatrix_trans(pack_f16x2(p0, p1));
        pb[t][1] = movmatrix_trans(pack_f16x2(p2, p3));
      }
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
            if (key < si.klo || key >= si.khi) ww[i >> 2] &= ~(0xFFu << (8 * (i & 3)));
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
    if (lane == 0) mbar_arrive(smem_addr(empty_bar + s));

    if (si.flags & kLast) {
      // ---- hand this warp's state for the segment to the epilogue ----
      float la = l_a, lb = l_b;
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        la += __shfl_xor_sync(0xffffffffu, la, off);
        lb += __shfl_xor_sync(0xffffffffu, lb, off);
      }
      if (!__all_sync(0xffffffffu, mbar_wait(smem_addr(slot_empty + slot), ((nslot / kSlots) & 1) ^ 1, abort_flag))) break;
      if (lane < 4) {
        mst[slot * kMaxGroup + 2 * c] = m_a;
        mst[slot * kMaxGroup + 2 * c + 1] = m_b;
        lst[slot * kMaxGroup + 2 * c] = la;
        lst[slot * kMaxGroup + 2 * c + 1] = lb;
      }
      if (lane == 0) slot_info[slot] = si;
      float* oa = ost + size_t(slot) * L::kSlotFloats + (2 * c) * L::kOStride;
      float* ob = oa + L::kOStride;
#pragma unroll
      for (int dt = 0; dt < KS; dt += 2) {
        // d-tiles dt, dt + 1: four consecutive dimensions
        int d;
        if constexpr (D == 128) d = 16 * r + 2 * dt;
        else d = dt < 4 ? 8 * r + 2 * dt : 64 + 4 * r;
        *reinterpret_cast<float4*>(oa + d) = make_float4(o[dt][0], o[dt][2], o[dt + 1][0], o[dt + 1][2]);
        *reinterpret_cast<float4*>(ob + d) = make_float4(o[dt][1], o[dt][3], o[dt + 1][1], o[dt + 1][3]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(slot_full + slot));
      ++nslot;
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
  int per_sm = 1;  // two CTAs per SM when they fit (shared memory grows with B)
  err = occupancy_blocks(&per_sm, fn, kThreads, bytes);
  if (err != cudaSuccess) return err;
  launch->grid = device_sm_count() * (per_sm >= kCtasPerSm ? kCtasPerSm : 1);
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
