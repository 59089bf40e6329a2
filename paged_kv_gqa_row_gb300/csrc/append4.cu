// The append into 4-bit pools for launches of many tokens (prompts): QK-norm,
// RoPE, quantization.  Launches of few tokens take append_rope.cu's split form.
//
// The results are append_rope.cu's, bit for bit: the float-pair evaluation of
// rope_math.cuh rounded once to bf16.  What it costs is avoided almost always:
// a lane first evaluates an output in float32, with the coefficients' low parts,
//     q = x2 s.hi + (x1 c.lo + x2 s.lo),  t = x1 c.hi + q   (fused products)
// and with a bound E on its error; where t - E and t + E round to the same bf16
// value, that is the answer, else (2 to 5 heads in a hundred have a lane near a
// border) the warp evaluates the head by the float pairs.  The bound, in units of
// 2^-24: q is rounded once (1 |q|), t once (1 |t|), the ends once (1 |t|), and
// what is of second order is below a quarter of (|q| + |t|): 3.5 max(|q|, |t|).
// With QK-norm the result is t r: the sum of D exact squares is rounded 7 times
// (two in the lane, five in the tree), the mean and eps add 3, half of it counts
// for r; r's own refinement 1.5, and the product 1: 8 more units of |t|, 11.5 in
// all (12 taken).
//
// A CTA takes one or two tokens, or half of one, with eight warps: its threads evaluate the
// sines and cosines once (one frequency of one token each), and after the one
// barrier every warp takes a share of one token's heads, the loads of the next two
// heads in flight while it works on two.  What bounds it: instructions, at 2.6 a cycle
// of an SM.  2048 tokens with QK-norm, 32 query heads on 8, D = 128: 10100 warp
// instructions a token, which launches of other shapes divide into 153 a query head
// (97 without the norm), 327 a key and value head (77 more where a pool scale is no
// power of two and the quantizer divides) and 2590 that a token costs whatever its heads
// (sines and cosines, and the coefficients, which each of its four warps sets up twice);
// 27 us (1.6 TB/s of what it reads and writes; 31 us with three CTAs an SM and four
// heads at once).
//
// Sources: as append_rope.cu; the 4-bit format is this library's (lnk_attn_desc).
#include "common.cuh"
#include "ptx.cuh"
#include "rope_math.cuh"

namespace lnk {
namespace {

using namespace rope;

constexpr int kWarps = 8;
constexpr int kHeadsAtOnce = 2;
constexpr int kMaxTokens = 2;    // of a CTA
constexpr int kCtasPerSm = 4;

// v in a range where none of the low parts below underflows, and no square of a
// head's larger elements (with room on both sides).
__device__ __forceinline__ bool rms_in_range(float v) { return v > 0x1p-90f && v < 0x1p100f; }

// The QK-norm factor 1 / sqrt(ss / D + eps) as a float pair (about 2^-44): one
// step from the float32 root r0.  With d = 1 - v r0^2 (v r0^2 in float pairs, the
// difference exact), 1 / sqrt(v) = r0 (1 + d / 2 + 3 d^2 / 8 + ...), |d| < 2^-20.
// (Double precision, as rope_math.cuh takes it once per head, is slow here: with
// it this kernel's FP64 pipe was a third of its time.)  A v out of range (norm_eps =
// 0 and tiny heads, or huge ones) is brought into it by a power of four.
template <int D>
__device__ __forceinline__ DF rms_factor_df(DF ss, float eps) {
  constexpr double kInv = 1.0 / D;
  constexpr float kHi = static_cast<float>(kInv), kLo = static_cast<float>(kInv - static_cast<double>(kHi));
  auto factor = [](DF sum, float e) {
    const DF v = df_add(df_mul(sum, DF{kHi, kLo}), DF{e, 0.f});
    const float r0 = rsqrtf(v.hi);
    const DF w = df_mul(v, two_prod(r0, r0));
    const float d = __fsub_rn(__fsub_rn(1.f, w.hi), w.lo);
    return fast_two_sum(r0, __fmul_rn(r0, __fmul_rn(d, __fmaf_rn(0.375f, d, 0.5f))));
  };
  const float size = __fmaf_rn(ss.hi, kHi, eps);
  if (!rms_in_range(size)) {
    const float four = size < 1.f ? 0x1p80f : 0x1p-60f, two = size < 1.f ? 0x1p40f : 0x1p-30f;
    const DF r = factor(DF{__fmul_rn(ss.hi, four), __fmul_rn(ss.lo, four)}, __fmul_rn(eps, four));
    return DF{ss.hi == 0.f && eps == 0.f ? INFINITY : __fmul_rn(r.hi, two), __fmul_rn(r.lo, two)};
  }
  return factor(ss, eps);
}

// The float-pair evaluation of one head (a whole warp calls it).
template <int D>
__device__ __noinline__ uint2 rotate_exact(uint32_t xlo, uint32_t xhi, Coefs c0, Coefs c1, bool normed, float eps) {
  const Coefs c[2] = {c0, c1};
  DF r{1.f, 0.f};
  if (normed) r = rms_factor_df<D>(head_sumsq(xlo, xhi), eps);
  uint32_t lo, hi;
  rotate_pairs(xlo, xhi, c, 0, normed, r, lo, hi);
  return make_uint2(lo, hi);
}

__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A coefficient of two neighbouring elements, as packed floats: high and low parts.
struct Pair {
  uint64_t hi, lo;
};

// Two outputs x a + y b (neighbouring elements), times r: their bf16 values (low
// half first).  `wrong` collects bits where the bounds round differently; emin: the
// least bound; esum: the bounds' sum (not finite if one of them is not, which it is
// where an output is not: q and t are NaN together, whatever x, y and r hold).
__device__ __forceinline__ uint32_t round_pair(uint64_t x, const Pair& a, uint64_t y, const Pair& b, uint64_t r,
                                               uint64_t unit, bool normed, uint32_t& wrong, float& emin, uint64_t& esum) {
  const uint64_t q = fma_f32x2(y, b.hi, fma_f32x2(y, b.lo, mul_f32x2(x, a.lo)));
  uint64_t t = fma_f32x2(x, a.hi, q);
  float q0, q1, t0, t1, e0, e1;
  f32x2_split(q, q0, q1);
  f32x2_split(t, t0, t1);
  const uint64_t e = mul_f32x2(f32x2(fmaxf(fabsf(q0), fabsf(t0)), fmaxf(fabsf(q1), fabsf(t1))), unit);
  if (normed) t = mul_f32x2(t, r);
  f32x2_split(e, e0, e1);
  emin = fmin3(emin, e0, e1);
  esum = add_f32x2(esum, e);
  float l0, l1, h0, h1;
  f32x2_split(fma_f32x2(e, f32x2(-1.f, -1.f), t), l0, l1);
  f32x2_split(add_f32x2(t, e), h0, h1);
  const uint32_t lo = pack_bf16x2(l0, l1), hi = pack_bf16x2(h0, h1);
  wrong |= lo ^ hi;
  return lo;
}

// POW2: both pool scales are powers of two (e2m1_pow2).
template <int D, bool POW2>
__global__ void __launch_bounds__(kWarps * 32, kCtasPerSm) append4_kernel(const AppendParams p) {
  constexpr int H = D / 2;
  __shared__ float4 s_angle[kMaxTokens][H];  // sine and cosine, as float pairs
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = p.splits;           // warps of a token
  const int parts = max(S / kWarps, 1);  // CTAs of a token
  const int tpc = max(kWarps / S, 1);    // tokens of the CTA
  const int t0 = static_cast<int>(blockIdx.x) / parts * tpc;
  // this warp: heads sp, sp + S, ... of token t
  const int t = t0 + warp / S, sp = static_cast<int>(blockIdx.x) % parts * kWarps + warp % S;
  const bool live = t < p.T;
  const bool has = lane < D / 4;    // lanes holding elements (e, e + 1) and (e + D/2, e + 1 + D/2)
  const int e = 2 * lane;

  // Before the wait: the angles and the slot (positions, rows, slots, table only).
  for (int i = tid; i < tpc * H; i += kWarps * 32) {
    const int ti = i / H, f = i % H;
    const int pos = t0 + ti < p.T ? p.positions[t0 + ti] : -1;
    if (pos < 0) continue;
    DF sn, cs;
    angle_sincos(pos, p.inv_freq[f], sn, cs);
    s_angle[ti][f] = make_float4(sn.hi, sn.lo, cs.hi, cs.lo);
  }
  const int pos = live ? p.positions[t] : -1;
  long long slot = -1;
  int bad = 0;
  if (pos >= 0) {
    if (p.slots != nullptr) {
      const int s = p.slots[t];
      if (s < 0 || static_cast<long long>(s) >= static_cast<long long>(p.num_pages) * kPage) bad = LNK_DEV_BAD_SLOT;
      else slot = s;
    } else {
      const int row = p.rows != nullptr ? p.rows[t] : t;
      if (row < 0 || row >= p.num_rows) {
        bad = LNK_DEV_BAD_ROW;
      } else if (pos >= p.pages_per_row * kPage) {
        bad = LNK_DEV_BAD_POSITION;
      } else {
        const int page = p.table[static_cast<long long>(row) * p.pages_per_row + pos / kPage];
        if (page < 0 || page >= p.num_pages) bad = LNK_DEV_BAD_PAGE;
        else slot = static_cast<long long>(page) * kPage + pos % kPage;
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  if (!live) return;
  if (bad && sp == 0 && lane == 0 && p.status != nullptr) atomicOr(p.status, bad);

  // sine and cosine of elements e, e + 1
  float4 an[2] = {make_float4(0.f, 0.f, 1.f, 0.f), make_float4(0.f, 0.f, 1.f, 0.f)};
  if (has && pos >= 0) {
    an[0] = s_angle[warp / S][e];
    an[1] = s_angle[warp / S][e + 1];
  }
  // The coefficients with the QK-norm weights: the queries', then the keys'.
  Coefs co[2];
  Pair c1, s2, c2, s1;  // of x1 and x2 in the low half's outputs, of x2 and x1 in the high half's
  auto set_weights = [&](const uint16_t* w) {
    float4 g = make_float4(1.f, 1.f, 1.f, 1.f);  // of elements e, e + 1, e + D/2, e + 1 + D/2
    if (w != nullptr && has) {
      const uint32_t a = *reinterpret_cast<const uint32_t*>(w + e), b = *reinterpret_cast<const uint32_t*>(w + H + e);
      g = make_float4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b));
    }
    co[0] = coefs_of(DF{an[0].x, an[0].y}, DF{an[0].z, an[0].w}, g.x, g.z);
    co[1] = coefs_of(DF{an[1].x, an[1].y}, DF{an[1].z, an[1].w}, g.y, g.w);
    c1 = {f32x2(co[0].gc1.hi, co[1].gc1.hi), f32x2(co[0].gc1.lo, co[1].gc1.lo)};
    s2 = {f32x2(-co[0].gs2.hi, -co[1].gs2.hi), f32x2(-co[0].gs2.lo, -co[1].gs2.lo)};
    c2 = {f32x2(co[0].gc2.hi, co[1].gc2.hi), f32x2(co[0].gc2.lo, co[1].gc2.lo)};
    s1 = {f32x2(co[0].gs1.hi, co[1].gs1.hi), f32x2(co[0].gs1.lo, co[1].gs1.lo)};
  };
  const float eps32 = static_cast<float>(p.norm_eps);

  uint8_t* kpage = reinterpret_cast<uint8_t*>(p.k_pool) + static_cast<size_t>(slot >= 0 ? slot / kPage : 0) * (36 * D);
  const size_t head_stride = static_cast<size_t>(p.num_pages) * (36 * D);
  const int j = slot >= 0 ? static_cast<int>(slot % kPage) : 0;
  const uint16_t* qrow = p.q + static_cast<size_t>(t) * p.hq * D + e;
  const uint16_t* krow = p.k + static_cast<size_t>(t) * p.hkv * D + e;
  uint16_t* orow = p.q_out + static_cast<size_t>(t) * p.hq * D + e;
  const bool reads = has && pos >= 0;
  // One head's rotated elements (zero for an inactive token).
  auto rotate = [&](uint32_t xl, uint32_t xh, bool normed, uint32_t& lo, uint32_t& hi) {
    lo = hi = 0u;
    if (pos < 0) return;
    const uint64_t x1 = f32x2(bf16_lo(xl), bf16_hi(xl)), x2 = f32x2(bf16_lo(xh), bf16_hi(xh));
    bool in_range = true;
    uint64_t r = 0, unit = f32x2(3.5f * 0x1p-24f, 3.5f * 0x1p-24f);
    if (normed) {
      float q0, q1;
      f32x2_split(fma_f32x2(x1, x1, mul_f32x2(x2, x2)), q0, q1);
      float ss = q0 + q1;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float v = __fadd_rn(__fmul_rn(ss, 1.f / D), eps32);
      const float r0 = rsqrtf(v);
      const float rr = __fmaf_rn(0.5f * r0, __fmaf_rn(-__fmul_rn(v, r0), r0, 1.f), r0);
      r = f32x2(rr, rr);
      unit = f32x2(12.f * 0x1p-24f * rr, 12.f * 0x1p-24f * rr);
      in_range = rms_in_range(v);  // (the bound counts no underflow)
    }
    uint32_t wrong = 0u;
    float emin = 1.f, es0, es1;
    uint64_t esum = 0;
    lo = round_pair(x1, c1, x2, s2, r, unit, normed, wrong, emin, esum);
    hi = round_pair(x2, c2, x1, s1, r, unit, normed, wrong, emin, esum);
    f32x2_split(esum, es0, es1);
    // (bounds that are zero, tiny, huge or NaN leave it to the float pairs)
    const bool certain = in_range && wrong == 0u && emin > 1e-30f && es0 + es1 < 1e30f;
    if (__any_sync(0xffffffffu, has && !certain)) {
      const uint2 x = rotate_exact<D>(xl, xh, co[0], co[1], normed, eps32);
      lo = x.x;
      hi = x.y;
    }
  };

  // ---- query heads ----
  uint32_t xlo[kHeadsAtOnce], xhi[kHeadsAtOnce];
  auto load = [&](const uint16_t* base, int heads, int h0, int u) {
    const int hh = h0 + S * u;
    xlo[u] = xhi[u] = 0u;
    if (hh < heads && reads) {
      xlo[u] = *reinterpret_cast<const uint32_t*>(base + hh * D);
      xhi[u] = *reinterpret_cast<const uint32_t*>(base + hh * D + H);
    }
  };
#pragma unroll
  for (int u = 0; u < kHeadsAtOnce; ++u) load(qrow, p.hq, sp, u);
  set_weights(p.q_norm_w);
#pragma unroll 1
  for (int h0 = sp; h0 < p.hq; h0 += S * kHeadsAtOnce) {
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int hh = h0 + S * u;
      if (hh >= p.hq) break;
      const uint32_t xl = xlo[u], xh = xhi[u];
      load(qrow, p.hq, h0 + S * kHeadsAtOnce, u);
      uint32_t lo, hi;
      rotate(xl, xh, p.q_norm_w != nullptr, lo, hi);
      if (has) {
        *reinterpret_cast<uint32_t*>(orow + hh * D) = lo;
        *reinterpret_cast<uint32_t*>(orow + hh * D + H) = hi;
      }
    }
  }
  if (slot < 0) return;
  // ---- key heads ----
#pragma unroll
  for (int u = 0; u < kHeadsAtOnce; ++u) load(krow, p.hkv, sp, u);
  set_weights(p.k_norm_w);
#pragma unroll 1
  for (int h0 = sp; h0 < p.hkv; h0 += S * kHeadsAtOnce) {
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int hh = h0 + S * u;
      if (hh >= p.hkv) break;
      const uint32_t xl = xlo[u], xh = xhi[u];
      load(krow, p.hkv, h0 + S * kHeadsAtOnce, u);
      uint32_t lo, hi;
      rotate(xl, xh, p.k_norm_w != nullptr, lo, hi);
      if (!has) lo = hi = 0u;
      store_key_e2m1<D, POW2>(kpage + static_cast<size_t>(hh) * head_stride, j, lane, has, lo, hi, p.k_scale);
    }
  }
  // ---- value heads, two at a time: lanes 0 .. 15 and 16 .. 31 ----
  uint8_t* vpage = reinterpret_cast<uint8_t*>(p.v_pool) + static_cast<size_t>(slot / kPage) * (36 * D);
  const int l = lane & 15;
#pragma unroll 2
  for (int v0 = 2 * sp; v0 < p.hkv; v0 += 2 * S) {
    const int vh = v0 + (lane >> 4);
    const bool mine = l < D / 8 && vh < p.hkv;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (mine) x = reinterpret_cast<const uint4*>(p.v + (static_cast<size_t>(t) * p.hkv + vh) * D)[l];
    store_value_e2m1<D, POW2>(vpage + static_cast<size_t>(vh) * head_stride, j, l, mine, x, p.v_scale);
  }
}

template <int D, bool POW2>
cudaError_t launch_t(const AppendParams& p, cudaStream_t stream) {
  const long long ctas = (static_cast<long long>(p.T) * p.splits + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append4_kernel<D, POW2>, p);
}

}  // namespace

// From half as many tokens as SMs on: below that append_rope.cu, which splits a
// token's heads over several CTAs (32 tokens, 32 query heads on 8, D = 128: 4.4 us
// against 5.5 here; 64 tokens: 5.5 and 5.4; 100 tokens: 7.3 and 5.0).
bool append4_takes(int tokens) { return 2 * static_cast<long long>(tokens) >= device_sm_count(); }

cudaError_t launch_append4(const AppendParams& p_in, int head_dim, cudaStream_t stream) {
  AppendParams p = p_in;
  // Warps of a token: two CTAs' as long as there are SMs for all tokens, then one CTA's,
  // then half of one.  With 16, 8 and 4 (us; 32 query heads on 8, D = 128 with QK-norm, and
  // 32 on 32, D = 96): 152 tokens 5.1, 5.6, 8.0 and 5.0, 5.8, 9.4; 304 tokens 7.6, 6.7, 8.4
  // and 8.2, 7.7, 9.6; 900 tokens 18.7, 15.0, 15.3 and 23.0, 19.5, 23.6; 1200 tokens 24.4,
  // 18.5, 16.4 and 30.5, 25.8, 24.6; 2048 tokens (the former) 33 with 8, 27 with 4.
  const int sms = device_sm_count();
  p.splits = p.T <= sms ? 2 * kWarps : p.T <= 7ll * sms ? kWarps : kWarps / 2;
  const bool pow2 = rope::e2m1_pow2(p.k_scale) && rope::e2m1_pow2(p.v_scale);
  switch (head_dim) {
    case 64: return pow2 ? launch_t<64, true>(p, stream) : launch_t<64, false>(p, stream);
    case 96: return pow2 ? launch_t<96, true>(p, stream) : launch_t<96, false>(p, stream);
    case 128: return pow2 ? launch_t<128, true>(p, stream) : launch_t<128, false>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
