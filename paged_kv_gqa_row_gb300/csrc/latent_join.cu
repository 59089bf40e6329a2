#include "latent.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

// Joins the partial sums of the units that the shares cut.  The blocks of all shares that
// start inside one unit (kJoinBlocks each) divide its rows by 128 numbers of a row: a warp
// takes such an item where the unit has up to kFewParts parts (every part's numbers are
// asked for before its weight is known), else a whole block, its warps the parts in turn.
// (What it takes is latency, and cold instruction caches: the end of the first kernel to
// the end of this one, 64 rows of 32 heads, 13 us with a list of the units and a warp a row.)
constexpr int kJoinThreads = 256;
constexpr int kJoinBlocks = 8;
constexpr int kFewParts = 8;

__device__ __forceinline__ void add_part(float4& acc, float f, const float4& x) {
  acc.x = fmaf(f, x.x, acc.x);
  acc.y = fmaf(f, x.y, acc.y);
  acc.z = fmaf(f, x.z, acc.z);
  acc.w = fmaf(f, x.w, acc.w);
}

// A part's weight 2^(its reference - the largest) (none has seen a key: 0)
__device__ __forceinline__ float part_weight(float mk, float m) { return mk == -INFINITY && m == -INFINITY ? 0.f : ex2_approx(mk - m); }

__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const __grid_constant__ LatentParams p) {
  __shared__ float4 s_acc[kJoinThreads];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, C = p.latent_dim;
  const int share = blockIdx.x / kJoinBlocks;
  const LatentCut cut = p.cuts[share];
  if (cut.j0 == 0) return;
  const long long p0 = share * cut.per - cut.j0;                     // the unit's first page in the stream
  const int c0 = static_cast<int>(p0 / cut.per) + 1;                 // first share that starts inside the unit
  const int cl = static_cast<int>((p0 + cut.np - 1) / cut.per);      // and the last
  const int parts = cl - c0 + 2;                                     // shares c0 - 1 .. cl
  const int nb = C / 128, items = cut.nt * p.heads * nb;
  const int blocks = (cl - c0 + 1) * kJoinBlocks, block = (share - c0) * kJoinBlocks + blockIdx.x % kJoinBlocks;
  const bool few = parts <= kFewParts;
  const int step = few ? blocks * (kJoinThreads / 32) : blocks;
  for (int i = few ? block * (kJoinThreads / 32) + warp : block; i < items; i += step) {
    const int r = i / nb, d = i % nb * 128 + lane * 4;
    const int hb = r / p.tile_rows, col = r % p.tile_rows;
    auto slot = [&](int k) {
      return (static_cast<size_t>(2 * (c0 - 1 + k) + (k == 0 ? 1 : 0)) * p.head_blocks + hb) * p.slot_rows + col;
    };
    float4 x[kFewParts];
    if (few) {
#pragma unroll
      for (int k = 0; k < kFewParts; ++k)
        if (k < parts) x[k] = *reinterpret_cast<const float4*>(p.o + slot(k) * C + d);
    }
    float m = -INFINITY, l = 0.f;
    float2 ml = make_float2(-INFINITY, 0.f);
    for (int k = lane; k < parts; k += 32) {
      ml = *reinterpret_cast<const float2*>(p.ml + slot(k) * 2);
      m = fmaxf(m, ml.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    for (int k = lane; k < parts; k += 32) {
      if (!few) ml = *reinterpret_cast<const float2*>(p.ml + slot(k) * 2);
      const float f = part_weight(ml.x, m);
      l += f == 0.f && ml.y == ml.y ? 0.f : f * ml.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    const float inv = l > 0.f ? 1.f / l : l;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (few) {
#pragma unroll
      for (int k = 0; k < kFewParts; ++k)
        if (k < parts) add_part(acc, part_weight(__shfl_sync(0xffffffffu, ml.x, k), m), x[k]);
    } else {
#pragma unroll 4
      for (int k = warp; k < parts; k += kJoinThreads / 32)
        add_part(acc, part_weight(p.ml[slot(k) * 2], m), *reinterpret_cast<const float4*>(p.o + slot(k) * C + d));
      s_acc[tid] = acc;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int w = 1; w < kJoinThreads / 32; ++w) add_part(acc, 1.f, s_acc[w * 32 + lane]);
      }
      __syncthreads();
    }
    if (few || warp == 0)
      *reinterpret_cast<uint2*>(p.out + (static_cast<size_t>(cut.t0) * p.heads + r) * C + d) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  }
}

}  // namespace

cudaError_t launch_latent_join(const LatentParams& p, cudaStream_t stream) {
  if (p.whole) return cudaSuccess;  // (no unit is cut)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(kJoinBlocks * p.teams));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_join_kernel, p);
}

}  // namespace lnk
