#include <algorithm>

#include "latent.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

// Joins the partial sums of the units that the shares cut.  The blocks of all shares that
// start inside one unit divide its rows: a warp takes a row, part after part, or a block 128
// numbers of a row, its warps the parts in turn (a long row's parts are as many as the
// shares), whichever ends first: 8 rows of 100 to 1500 keys and 64 heads, whose units have few
// blocks, 43 us with blocks from nine parts on, 21 us so.
// What a launch takes is latency and cold instruction caches, so the
// first numbers are asked for before their weights are known, and the blocks are so few and
// small that all are on the SMs when the first kernel ends.  Both kernels, decode of 32
// rows of 128 heads, 64 rows of 32, 2 long rows of 40: eight small blocks a share, a warp
// for 128 numbers of a row, 63.6, 71.2 and 62.9 us; 4 blocks an SM 59.6, 75.0 and 69.7; these 2
// an SM 56.8, 68.6 and 64.2; one 63.6, 71.0 and 65.7; 16 parts of a warp at once 64.4, 72.9, 68.7;
// a third form, a warp for 128 numbers, beside these two 57.4, 74.9 and 80.
constexpr int kJoinThreads = 256;
constexpr int kJoinCtasPerSm = 2;
constexpr int kBlockItem = 4;  // what a block's 128 numbers take, in parts of a warp's row
constexpr int kAtOnce = 12;  // parts a warp of a block has under way

__device__ __forceinline__ void add_part(float4& acc, float f, const float4& x) {
  acc.x = fmaf(f, x.x, acc.x);
  acc.y = fmaf(f, x.y, acc.y);
  acc.z = fmaf(f, x.z, acc.z);
  acc.w = fmaf(f, x.w, acc.w);
}

// A part's weight 2^(its reference - the largest) (none has seen a key: 0)
__device__ __forceinline__ float part_weight(float mk, float m) { return mk == -INFINITY && m == -INFINITY ? 0.f : ex2_approx(mk - m); }

__global__ void __launch_bounds__(kJoinThreads, kJoinCtasPerSm)
    latent_join_kernel(const __grid_constant__ LatentParams p, int per_share) {
  __shared__ float4 s_acc[kJoinThreads];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, C = p.latent_dim;
  const int share = blockIdx.x / per_share;
  const LatentCut cut = p.cuts[share];
  if (cut.j0 == 0) return;
  const long long p0 = share * cut.per - cut.j0;                     // the unit's first page in the stream
  const int c0 = static_cast<int>(p0 / cut.per) + 1;                 // first share that starts inside the unit
  const int cl = static_cast<int>((p0 + cut.np - 1) / cut.per);      // and the last
  const int parts = cl - c0 + 2;                                     // shares c0 - 1 .. cl
  const int nb = C / 128, rows = cut.nt * p.heads;
  const int blocks = (cl - c0 + 1) * per_share, block = (share - c0) * per_share + static_cast<int>(blockIdx.x) % per_share;
  const bool few = parts <= 32 && (rows + 8 * blocks - 1) / (8 * blocks) * parts <= (rows * nb + blocks - 1) / blocks * kBlockItem;
  const int items = few ? rows : rows * nb, step = few ? blocks * (kJoinThreads / 32) : blocks;
  for (int i = few ? block * (kJoinThreads / 32) + warp : block; i < items; i += step) {
    const int r = few ? i : i / nb, d = (few ? 0 : i % nb * 128) + lane * 4;
    const int hb = r / p.tile_rows, col = r % p.tile_rows;
    auto slot = [&](int k) {
      return (static_cast<size_t>(2 * (c0 - 1 + k) + (k == 0 ? 1 : 0)) * p.head_blocks + hb) * p.slot_rows + col;
    };
    // numbers d .. + 3 of part k, + 128 j
    auto part = [&](int k, int j) { return *reinterpret_cast<const float4*>(p.o + slot(k) * C + d + 128 * j); };
    float4 x[kAtOnce];
    if (few) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < nb) x[j] = part(0, j);
    } else {
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (warp + 8 * k < parts) x[k] = part(warp + 8 * k, 0);
    }
    // the parts' references and sums: the largest reference, the whole sum
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
    uint16_t* out = p.out + (static_cast<size_t>(cut.t0) * p.heads + r) * C + d;
    auto store = [&](int j, const float4& a) {
      *reinterpret_cast<uint2*>(out + 128 * j) =
          make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    };
    if (few) {
      float4 acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
      for (int k = 0; k < parts; ++k) {
        const float f = part_weight(__shfl_sync(0xffffffffu, ml.x, k), m);
        float4 y[4];  // the next part's, asked for first
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nb && k + 1 < parts) y[j] = part(k + 1, j);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nb) {
            add_part(acc[j], f, x[j]);
            x[j] = y[j];
          }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < nb) store(j, acc[j]);
    } else {
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (warp + 8 * k < parts) add_part(acc, part_weight(p.ml[slot(warp + 8 * k) * 2], m), x[k]);
#pragma unroll 4
      for (int k = warp + 8 * kAtOnce; k < parts; k += 8) add_part(acc, part_weight(p.ml[slot(k) * 2], m), part(k, 0));
      s_acc[tid] = acc;
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int w = 1; w < kJoinThreads / 32; ++w) add_part(acc, 1.f, s_acc[w * 32 + lane]);
        store(0, acc);
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_latent_join(const LatentParams& p, cudaStream_t stream) {
  if (p.whole) return cudaSuccess;  // (no unit is cut)
  cudaLaunchConfig_t cfg = {};
  const int per_share = std::max(1, kJoinCtasPerSm * device_sm_count() / p.teams);
  cfg.gridDim = dim3(static_cast<unsigned>(per_share * p.teams));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_join_kernel, p, per_share);
}

}  // namespace lnk
