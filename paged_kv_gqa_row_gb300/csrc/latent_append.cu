// lnk_latent_append: per token, the latent vector's RMS norm, the rotation of the key's
// and the query heads' last R numbers, and the write of [c, k] into the token's place.
//
// A token's heads are split over S CTAs of 128 threads (S = 1 for launches of many
// tokens); the first also takes the token's row: up to four numbers of c a thread.  Every
// stored number is rounded once, to bf16: in float32 where its error bound leaves no doubt
// about that rounding, else from the float-pair arithmetic of rope_math.cuh, in which the
// norm's sum of squares and factor are computed throughout.
//
// Bound: one chain of dependent reads for few tokens (64 tokens of 64 heads: 2.9 us), the issue
// of instructions for many (2000 tokens of 40 heads, 27 MB: 11.0 us, 1100 a warp; 4.05 at the
// copy rate).
#include <algorithm>

#include "latent.cuh"
#include "rope_math.cuh"

namespace lnk {
namespace {

using namespace rope;

constexpr int kThreads = 128;
constexpr int kCtasPerSm = 4;     // launches of few tokens aim at this many CTAs per SM
constexpr int kHeadsPerCta = 8;   // and give each at least this many heads

__device__ __forceinline__ DF add_pair(DF a, float hi, float lo) {
  const DF w = two_sum(a.hi, hi);
  return two_sum(w.hi, __fadd_rn(w.lo, __fadd_rn(a.lo, lo)));
}

// The norm's factor 1 / sqrt(ss / C + eps): a float32 estimate and one Newton step on float
// pairs, good to 2^-42; sums whose mean square is tiny or huge go through double precision.
__device__ __forceinline__ DF norm_factor(DF ss, const LatentAppendParams& p) {
  const DF v = add_pair(df_mul(ss, DF{p.inv_dim[0], p.inv_dim[1]}), p.eps[0], p.eps[1]);
  if (!(v.hi > 1e-18f && v.hi < 1e18f)) return rms_factor(ss, p.latent_dim, p.norm_eps);
  const float r0 = rsqrtf(v.hi);
  const DF vr = df_mul(v, two_prod(r0, r0));              // v r0^2 = 1 + e, |e| about 2^-22
  const float e = __fadd_rn(__fadd_rn(vr.hi, -1.f), vr.lo);
  return fast_two_sum(r0, __fmul_rn(__fmul_rn(-0.5f, r0), e));
}

// Two numbers to bf16 in one rounding where float32 says which way: each is off by at most
// `el`, `eh`; false where one of them may round either way (or is not finite).
__device__ __forceinline__ bool sure_bf16x2(float lo, float hi, float el, float eh, uint32_t& bits) {
  bits = floats_to_bf16x2(__fadd_rn(lo, el), __fadd_rn(hi, eh));
  return bits == floats_to_bf16x2(__fsub_rn(lo, el), __fsub_rn(hi, eh));
}

// x w r of two neighbours (x, w bf16 values, whose product is exact).
__device__ __forceinline__ uint32_t normed(uint32_t x, uint32_t w, DF r) {
  const float a = __fmul_rn(bf16_lo(x), bf16_lo(w)), b = __fmul_rn(bf16_hi(x), bf16_hi(w));
  const float ar = __fmul_rn(a, r.hi), br = __fmul_rn(b, r.hi);
  uint32_t bits;
  // (the product's rounding and r's low part: 2^-23 together)
  if (sure_bf16x2(ar, br, __fmul_rn(fabsf(ar), 0x1p-21f), __fmul_rn(fabsf(br), 0x1p-21f), bits)) return bits;
  const float c = df_off_tie(mul_df(DF{a, 0.f}, r)), d = df_off_tie(mul_df(DF{b, 0.f}, r));
  return floats_to_bf16x2(c == c ? c : ar, d == d ? d : br);
}

// rotate_pairs (without a factor), in float32 where that decides the rounding: sine and
// cosine, the two products and their sum are off by at most 2.5 2^-23 of |x1| + |x2|
// together, and one element in a thousand is too near a tie.
// (quick: cosine and sine of elements e and e + 1 in float32)
__device__ __forceinline__ void rotate(uint32_t xlo, uint32_t xhi, const Coefs* c, float4 quick, int e, uint32_t& lo_bits,
                                       uint32_t& hi_bits) {
  float o1[2], o2[2], err[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float cs = k ? quick.z : quick.x, sn = k ? quick.w : quick.y;
    const float x1 = k ? bf16_hi(xlo) : bf16_lo(xlo), x2 = k ? bf16_hi(xhi) : bf16_lo(xhi);
    o1[k] = __fmaf_rn(x1, cs, -__fmul_rn(x2, sn));
    o2[k] = __fmaf_rn(x2, cs, __fmul_rn(x1, sn));
    err[k] = __fmul_rn(__fadd_rn(fabsf(x1), fabsf(x2)), 0x1p-21f);
  }
  if (sure_bf16x2(o1[0], o1[1], err[0], err[1], lo_bits) & sure_bf16x2(o2[0], o2[1], err[0], err[1], hi_bits)) return;
  rotate_pairs(xlo, xhi, c, e, false, DF{1.f, 0.f}, lo_bits, hi_bits);
}

template <int R>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const __grid_constant__ LatentAppendParams p, int splits) {
  constexpr int H = R / 2, kLanes = R / 4;  // threads of a head: two numbers of each half
  __shared__ Coefs s_coef[H];
  __shared__ __align__(16) float2 s_quick[H];
  __shared__ DF s_ss[kThreads / 32];
  __shared__ long long s_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int t = blockIdx.x / splits, sp = blockIdx.x % splits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int pos = p.positions[t];
  // before the wait for the kernel before this one: positions, rows, slots and the table only
  DF sn{0.f, 0.f}, cs{0.f, 0.f};
  if (tid < H && pos >= 0) angle_sincos(pos, p.inv_freq[tid], sn, cs);
  int bad = 0;
  if (tid == kThreads - 1) {
    long long slot = -1;
    if (pos >= 0 && sp == 0) {
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
    s_slot = slot;
  }

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bad && p.status != nullptr) atomicOr(p.status, bad);
  // ---- loads ----
  const int C = p.latent_dim, W = C + R;
  const uint16_t* row_in = p.kv + static_cast<size_t>(t) * W;
  uint2 x = make_uint2(0u, 0u), w = make_uint2(0x3F803F80u, 0x3F803F80u);  // (bf16 ones)
  const bool has = sp == 0 && 4 * tid < C;
  if (has && pos >= 0) {
    x = *reinterpret_cast<const uint2*>(row_in + 4 * tid);
    if (p.norm_w != nullptr) w = *reinterpret_cast<const uint2*>(p.norm_w + 4 * tid);
  }
  const int e = 2 * (tid % kLanes);
  constexpr int kBatch = 2;  // heads whose loads are in flight together
  const int hstep = splits * (kThreads / kLanes);
  uint32_t xlo[kBatch], xhi[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * hstep;
      xlo[k] = xhi[k] = 0u;
      if (h < p.heads && pos >= 0) {
        const uint16_t* src = p.q + (static_cast<size_t>(t) * p.heads + h) * p.q_stride + e;
        xlo[k] = *reinterpret_cast<const uint32_t*>(src);
        xhi[k] = *reinterpret_cast<const uint32_t*>(src + H);
      }
    }
  };
  load(sp + splits * (tid / kLanes));
  if (tid < H) {
    s_coef[tid] = coefs_of(sn, cs, 1.f, 1.f);
    s_quick[tid] = make_float2(cs.hi, sn.hi);
  }
  if (sp == 0 && p.norm_w != nullptr) {
    const float a0 = bf16_lo(x.x), a1 = bf16_hi(x.x), a2 = bf16_lo(x.y), a3 = bf16_hi(x.y);
    DF acc = two_sum(__fmul_rn(a0, a0), __fmul_rn(a1, a1));
    const DF u = two_sum(__fmul_rn(a2, a2), __fmul_rn(a3, a3));
    acc = add_pair(acc, u.hi, u.lo);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float oh = __shfl_xor_sync(0xffffffffu, acc.hi, o), ol = __shfl_xor_sync(0xffffffffu, acc.lo, o);
      acc = add_pair(acc, oh, ol);
    }
    if (lane == 0) s_ss[warp] = acc;
  }
  __syncthreads();
  // ---- query heads of this CTA ----
  const float4 quick = *reinterpret_cast<const float4*>(&s_quick[e]);
  for (int h0 = sp + splits * (tid / kLanes); h0 < p.heads;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int h = h0 + k * hstep;
      if (h >= p.heads) break;
      uint32_t lo = 0u, hi = 0u;
      if (pos >= 0) rotate(xlo[k], xhi[k], s_coef, quick, e, lo, hi);
      uint16_t* dst = p.q_out + (static_cast<size_t>(t) * p.heads + h) * p.q_out_stride + e;
      *reinterpret_cast<uint32_t*>(dst) = lo;
      *reinterpret_cast<uint32_t*>(dst + H) = hi;
    }
    h0 += kBatch * hstep;
    if (h0 < p.heads) load(h0);
  }
  if (sp != 0) return;
  // ---- the token's row ----
  DF r{1.f, 0.f};
  if (p.norm_w != nullptr) {
    DF ss = s_ss[0];
    for (int k = 1; k < kThreads / 32; ++k) ss = add_pair(ss, s_ss[k].hi, s_ss[k].lo);
    r = norm_factor(ss, p);
  }
  uint16_t* pool_row = s_slot >= 0 ? p.pool + static_cast<size_t>(s_slot) * W : nullptr;
  uint16_t* kv_row = p.kv_out != nullptr ? p.kv_out + static_cast<size_t>(t) * W : nullptr;
  if (has) {
    uint2 c = x;
    if (p.norm_w != nullptr && pos >= 0) {
      c.x = normed(x.x, w.x, r);
      c.y = normed(x.y, w.y, r);
    }
    if (pool_row != nullptr) *reinterpret_cast<uint2*>(pool_row + 4 * tid) = c;
    if (kv_row != nullptr) *reinterpret_cast<uint2*>(kv_row + 4 * tid) = c;
  }
  if (tid < kLanes) {
    uint32_t lo = 0u, hi = 0u;
    if (pos >= 0)
      rotate(*reinterpret_cast<const uint32_t*>(row_in + C + e), *reinterpret_cast<const uint32_t*>(row_in + C + H + e), s_coef,
             quick, e, lo, hi);
    if (pool_row != nullptr) {
      *reinterpret_cast<uint32_t*>(pool_row + C + e) = lo;
      *reinterpret_cast<uint32_t*>(pool_row + C + H + e) = hi;
    }
    if (kv_row != nullptr) {
      *reinterpret_cast<uint32_t*>(kv_row + C + e) = lo;
      *reinterpret_cast<uint32_t*>(kv_row + C + H + e) = hi;
    }
  }
}

template <int R>
cudaError_t launch_t(const LatentAppendParams& p, cudaStream_t stream) {
  const cudaError_t carve = prefer_max_shared(reinterpret_cast<const void*>(latent_append_kernel<R>));
  if (carve != cudaSuccess) return carve;
  const long long sms = device_sm_count();
  const int splits = static_cast<int>(std::max<long long>(
      1, std::min<long long>((p.heads + kHeadsPerCta - 1) / kHeadsPerCta, kCtasPerSm * sms / p.T)));
  const long long ctas = static_cast<long long>(p.T) * splits;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_append_kernel<R>, p, splits);
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendParams& p, cudaStream_t stream) {
  return p.rope_dim == 64 ? launch_t<64>(p, stream) : launch_t<32>(p, stream);
}

}  // namespace lnk
