// lnk_latent_append: per token, the latent vector's RMS norm, the rotation of the key's
// and the query heads' last R numbers, and the write of [c, k] into the token's place.
//
// A token's heads are split over S CTAs of 128 threads (S = 1 for launches of many
// tokens); the first also takes the token's row: up to four numbers of c a thread.  The
// rotation is the float-pair arithmetic of rope_math.cuh; the norm's sum of squares is
// a float pair too, its factor is computed once a token in double precision, and every
// stored number is rounded once, to bf16.
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

// x w r to the nearest bf16's float (x, w bf16 values; their product is exact).
__device__ __forceinline__ float normed(float x, float w, DF r) {
  const float xw = __fmul_rn(x, w);
  const float v = df_off_tie(mul_df(DF{xw, 0.f}, r));
  return v == v ? v : __fmul_rn(xw, r.hi);
}

template <int R>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const __grid_constant__ LatentAppendParams p, int splits) {
  constexpr int H = R / 2, kLanes = R / 4;  // threads of a head: two numbers of each half
  __shared__ Coefs s_coef[H];
  __shared__ DF s_ss[kThreads / 32];
  __shared__ DF s_r;
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
  if (tid < H) s_coef[tid] = coefs_of(sn, cs, 1.f, 1.f);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (bad && p.status != nullptr) atomicOr(p.status, bad);
  const int C = p.latent_dim, W = C + R;
  const uint16_t* row_in = p.kv + static_cast<size_t>(t) * W;
  uint2 x = make_uint2(0u, 0u), w = make_uint2(0x3F803F80u, 0x3F803F80u);  // (bf16 ones)
  const bool has = sp == 0 && 4 * tid < C;
  if (has && pos >= 0) {
    x = *reinterpret_cast<const uint2*>(row_in + 4 * tid);
    if (p.norm_w != nullptr) w = *reinterpret_cast<const uint2*>(p.norm_w + 4 * tid);
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
  const int e = 2 * (tid % kLanes);
  for (int h = sp + splits * (tid / kLanes); h < p.heads; h += splits * (kThreads / kLanes)) {
    const uint16_t* src = p.q + (static_cast<size_t>(t) * p.heads + h) * p.q_stride;
    uint16_t* dst = p.q_out + (static_cast<size_t>(t) * p.heads + h) * p.q_out_stride;
    uint32_t lo = 0u, hi = 0u;
    if (pos >= 0)
      rotate_pairs(*reinterpret_cast<const uint32_t*>(src + e), *reinterpret_cast<const uint32_t*>(src + H + e), s_coef, e,
                   false, DF{1.f, 0.f}, lo, hi);
    *reinterpret_cast<uint32_t*>(dst + e) = lo;
    *reinterpret_cast<uint32_t*>(dst + H + e) = hi;
  }
  if (sp != 0) return;
  // ---- the token's row ----
  DF r{1.f, 0.f};
  if (p.norm_w != nullptr) {
    if (tid == 0) {
      DF ss = s_ss[0];
      for (int k = 1; k < kThreads / 32; ++k) ss = add_pair(ss, s_ss[k].hi, s_ss[k].lo);
      s_r = rms_factor(ss, C, p.norm_eps);
    }
    __syncthreads();
    r = s_r;
  }
  uint16_t* pool_row = s_slot >= 0 ? p.pool + static_cast<size_t>(s_slot) * W : nullptr;
  uint16_t* kv_row = p.kv_out != nullptr ? p.kv_out + static_cast<size_t>(t) * W : nullptr;
  if (has) {
    uint2 c = x;
    if (p.norm_w != nullptr && pos >= 0) {
      c.x = floats_to_bf16x2(normed(bf16_lo(x.x), bf16_lo(w.x), r), normed(bf16_hi(x.x), bf16_hi(w.x), r));
      c.y = floats_to_bf16x2(normed(bf16_lo(x.y), bf16_lo(w.y), r), normed(bf16_hi(x.y), bf16_hi(w.y), r));
    }
    if (pool_row != nullptr) *reinterpret_cast<uint2*>(pool_row + 4 * tid) = c;
    if (kv_row != nullptr) *reinterpret_cast<uint2*>(kv_row + 4 * tid) = c;
  }
  if (tid < kLanes) {
    uint32_t lo = 0u, hi = 0u;
    if (pos >= 0)
      rotate_pairs(*reinterpret_cast<const uint32_t*>(row_in + C + e), *reinterpret_cast<const uint32_t*>(row_in + C + H + e),
                   s_coef, e, false, DF{1.f, 0.f}, lo, hi);
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
