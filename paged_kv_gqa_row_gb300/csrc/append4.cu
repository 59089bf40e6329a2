// The append into 4-bit pools for launches of many tokens (prompts): QK-norm,
// RoPE, quantization.  Launches of few tokens take append_rope.cu's split form.
//
// The results are append_rope.cu's, bit for bit: the float-pair evaluation of
// rope_math.cuh rounded once to bf16.  What it costs is avoided almost always:
// a lane first evaluates its outputs in float32 with a bound E on the error,
//     |u - exact| <= E,   E = 2^-21 S (2^-20 S r with QK-norm),
//     S = |x1 c1| + |x2 s2|, the two terms of the rotation, r the RMS factor,
// and where u - E and u + E round to the same bf16 value, that is the answer.
// Otherwise (about one head in ten: some lane of the warp is near a border) the
// warp evaluates the head by the float pairs.  The bound: each coefficient is
// rounded once or twice (cosine or sine to float32, times the weight), each
// product and the sum once: at most 4 S units of 2^-24.  With QK-norm the
// float32 sum of the 128 exact squares adds at most 9 units to the mean's
// relative error, half of that to r, the reciprocal root at most 4 and the last
// product 1; u - E and u + E are rounded too: 5 units without, 15.5 with the norm,
// against 8 and 16 in E.
//
// A warp works alone, without barriers: it takes one token (or one of S shares
// of its heads), each lane evaluates the sine and cosine of its two frequencies
// in registers, and the loads of four heads are in flight together.  What bounds
// it: instructions (about 70 a head, 330 a frequency, 10 a division of the
// quantizer).
//
// Sources: as append_rope.cu; the 4-bit format is this library's (lnk_attn_desc).
#include <algorithm>

#include "common.cuh"
#include "ptx.cuh"
#include "rope_math.cuh"

namespace lnk {
namespace {

using namespace rope;

constexpr int kWarps = 8;
constexpr int kHeadsAtOnce = 4;
constexpr int kWarpsPerSm = 24;  // what a launch aims at

// The float-pair evaluation of one head (a whole warp calls it).
template <int D>
__device__ __noinline__ uint2 rotate_exact(uint32_t xlo, uint32_t xhi, DF sn0, DF cs0, DF sn1, DF cs1, float4 g,
                                           bool normed, double eps) {
  const Coefs c[2] = {coefs_of(sn0, cs0, g.x, g.z), coefs_of(sn1, cs1, g.y, g.w)};
  DF r{1.f, 0.f};
  if (normed) r = rms_factor(head_sumsq(xlo, xhi), D, eps);
  uint32_t lo, hi;
  rotate_pairs(xlo, xhi, c, 0, normed, r, lo, hi);
  return make_uint2(lo, hi);
}

// One output and whether it is certain.
__device__ __forceinline__ uint32_t round_certain(float u, float e, bool& certain) {
  const uint32_t w = pack_bf16x2(__fsub_rn(u, e), __fadd_rn(u, e));
  // (zero, tiny, huge and NaN bounds go the other way)
  certain = certain && (w >> 16) == (w & 0xFFFFu) && e > 1e-30f && e < 1e30f;
  return w & 0xFFFFu;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) append4_kernel(const AppendParams p) {
  constexpr int H = D / 2;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = p.splits;
  const long long gw = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const int t = static_cast<int>(gw / S), sp = static_cast<int>(gw % S);  // token; heads sp, sp + S, ...
  const bool live = t < p.T;
  const bool has = lane < D / 4;  // lanes holding elements (e, e + 1) and (e + D/2, e + 1 + D/2)
  const int e = 2 * lane;

  // Before the wait: the slot and the angles (positions, rows, slots, table only).
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
  DF sn[2] = {{0.f, 0.f}, {0.f, 0.f}}, cs[2] = {{1.f, 0.f}, {1.f, 0.f}};
  if (has && pos >= 0) {
#pragma unroll
    for (int k = 0; k < 2; ++k) angle_sincos(pos, p.inv_freq[e + k], sn[k], cs[k]);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  if (bad && sp == 0 && lane == 0 && p.status != nullptr) atomicOr(p.status, bad);

  // QK-norm weights of elements e, e + 1, e + D/2, e + 1 + D/2: queries, keys
  float4 gam[2] = {make_float4(1.f, 1.f, 1.f, 1.f), make_float4(1.f, 1.f, 1.f, 1.f)};
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint16_t* g = w == 0 ? p.q_norm_w : p.k_norm_w;
    if (g != nullptr && has) {
      const uint32_t a = *reinterpret_cast<const uint32_t*>(g + e), b = *reinterpret_cast<const uint32_t*>(g + H + e);
      gam[w] = make_float4(bf16_lo(a), bf16_hi(a), bf16_lo(b), bf16_hi(b));
    }
  }
  const float eps32 = static_cast<float>(p.norm_eps);

  // ---- rotated heads: queries, then keys ----
  const int nrot = p.hq + p.hkv;
  uint8_t* kpage = reinterpret_cast<uint8_t*>(p.k_pool) + static_cast<size_t>(slot >= 0 ? slot / kPage : 0) * (36 * D);
  const size_t head_stride = static_cast<size_t>(p.num_pages) * (36 * D);
  const int j = slot >= 0 ? static_cast<int>(slot % kPage) : 0;
#pragma unroll 1
  for (int h0 = sp; h0 < nrot; h0 += S * kHeadsAtOnce) {
    uint32_t xlo[kHeadsAtOnce], xhi[kHeadsAtOnce];
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int hh = h0 + S * u;
      xlo[u] = xhi[u] = 0u;
      if (hh < nrot && has && pos >= 0) {
        const uint16_t* src = hh < p.hq ? p.q + (static_cast<size_t>(t) * p.hq + hh) * D
                                        : p.k + (static_cast<size_t>(t) * p.hkv + (hh - p.hq)) * D;
        xlo[u] = *reinterpret_cast<const uint32_t*>(src + e);
        xhi[u] = *reinterpret_cast<const uint32_t*>(src + H + e);
      }
    }
#pragma unroll
    for (int u = 0; u < kHeadsAtOnce; ++u) {
      const int hh = h0 + S * u;
      if (hh >= nrot) break;
      const bool is_q = hh < p.hq;
      if (!is_q && slot < 0) continue;
      uint32_t lo = 0u, hi = 0u;  // (an inactive token's queries are zero)
      if (pos >= 0) {
        const float4 g = gam[is_q ? 0 : 1];
        const bool normed = (is_q ? p.q_norm_w : p.k_norm_w) != nullptr;
        const float x1[2] = {bf16_lo(xlo[u]), bf16_hi(xlo[u])}, x2[2] = {bf16_lo(xhi[u]), bf16_hi(xhi[u])};
        float r = 1.f, unit = 0x1p-21f;
        if (normed) {
          float ss = fmaf(x1[0], x1[0], x1[1] * x1[1]) + fmaf(x2[0], x2[0], x2[1] * x2[1]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          r = rsqrtf(ss * (1.f / D) + eps32);
          unit = 0x1p-20f * r;
        }
        bool certain = true;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float g1 = k ? g.y : g.x, g2 = k ? g.w : g.z;
          const float a = x1[k] * (g1 * cs[k].hi), b = x2[k] * (g2 * sn[k].hi);
          const float c = x2[k] * (g2 * cs[k].hi), d = x1[k] * (g1 * sn[k].hi);
          lo |= round_certain((a - b) * r, (fabsf(a) + fabsf(b)) * unit, certain) << (16 * k);
          hi |= round_certain((c + d) * r, (fabsf(c) + fabsf(d)) * unit, certain) << (16 * k);
        }
        if (__any_sync(0xffffffffu, has && !certain)) {
          const uint2 x = rotate_exact<D>(xlo[u], xhi[u], sn[0], cs[0], sn[1], cs[1], g, normed, p.norm_eps);
          lo = x.x;
          hi = x.y;
        }
        if (!has) lo = hi = 0u;
      }
      if (is_q) {
        if (has) {
          uint16_t* dst = p.q_out + (static_cast<size_t>(t) * p.hq + hh) * D;
          *reinterpret_cast<uint32_t*>(dst + e) = lo;
          *reinterpret_cast<uint32_t*>(dst + H + e) = hi;
        }
      } else {
        store_key_e2m1<D>(kpage + static_cast<size_t>(hh - p.hq) * head_stride, j, lane, has, lo, hi, p.k_scale);
      }
    }
  }
  if (slot < 0) return;
  // ---- value heads, two at a time: lanes 0 .. 15 and 16 .. 31 ----
  uint8_t* vpage = reinterpret_cast<uint8_t*>(p.v_pool) + static_cast<size_t>(slot / kPage) * (36 * D);
  const int l = lane & 15;
#pragma unroll 2
  for (int v0 = 2 * sp; v0 < p.hkv; v0 += 2 * S) {
    const int vh = v0 + (lane >> 4);
    const bool mine = l < D / 8 && vh < p.hkv;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (mine) x = reinterpret_cast<const uint4*>(p.v + (static_cast<size_t>(t) * p.hkv + vh) * D)[l];
    store_value_e2m1<D>(vpage + static_cast<size_t>(vh) * head_stride, j, l, mine, x, p.v_scale);
  }
}

template <int D>
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
  return cudaLaunchKernelEx(&cfg, append4_kernel<D>, p);
}

}  // namespace

bool append4_takes(int tokens) { return tokens >= device_sm_count(); }

cudaError_t launch_append4(const AppendParams& p_in, int head_dim, cudaStream_t stream) {
  AppendParams p = p_in;
  // enough warps for kWarpsPerSm on every SM, a batch of heads for each at least
  const long long want = (static_cast<long long>(kWarpsPerSm) * device_sm_count() + p.T - 1) / p.T;
  const int most = std::max(1, (p.hq + p.hkv) / kHeadsAtOnce);
  p.splits = static_cast<int>(std::max<long long>(1, std::min<long long>(most, want)));
  switch (head_dim) {
    case 64: return launch_t<64>(p, stream);
    case 96: return launch_t<96>(p, stream);
    case 128: return launch_t<128>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
