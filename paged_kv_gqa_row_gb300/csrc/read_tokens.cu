// lnk_paged_read_tokens: the stored keys and values of given tokens as bf16,
// for every pool type (the append's inverse).
//
// One thread per 8 elements of one (token, kv head), in both pools: it reads 16
// bytes of a bf16 pool, 8 of an 8-bit pool, or 4 code bytes and one scale byte of a
// 4-bit pool, and stores 16 bytes.  The elements of a token's heads are
// consecutive threads, so the stores are whole lines; the loads of one head are
// one contiguous row of its page.  Bound by latency (position, table, page): 2048
// tokens of 8 heads, D = 128, 4-bit pools, 2.9 us in a row of calls, 3.6 TB/s of what
// it reads and writes, most of it in L2 (8.6 us with a thread per pool and 64-bit
// division throughout).
#include <cuda_fp8.h>

#include "common.cuh"
#include "ptx.cuh"

namespace lnk {
namespace {

constexpr int kThreads = 256;

// Eight values of a row, packed in pairs (low half first).
template <int D, int KV>
__device__ __forceinline__ uint4 read8(const uint8_t* page, int j, int e8, float scale) {
  if constexpr (KV == LNK_KV_BF16) {
    return reinterpret_cast<const uint4*>(page + static_cast<size_t>(j) * (2 * D))[e8];
  } else {
    uint32_t h[4];  // f16 pairs: the codes' values, times the block's scale for E2M1 (both exact)
    if constexpr (KV == LNK_KV_E4M3) {
      const uint2 w = reinterpret_cast<const uint2*>(page + j * D)[e8];
      e4m3x4_to_f16x2x2(w.x, h[0], h[1]);
      e4m3x4_to_f16x2x2(w.y, h[2], h[3]);
    } else {
      const uint32_t w = reinterpret_cast<const uint32_t*>(page + j * (D / 2))[e8];
      const uint32_t s = page[32 * D + ((j & 3) * (D / 16) + (e8 >> 1)) * 16 + (j >> 2)];
      e2m1x8_to_f16x2x4(w, h);
      const uint32_t s2 = e4m3x2_to_f16x2(s | (s << 8));
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = mul_f16x2(h[i], s2);
    }
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
      r[i] = pack_bf16x2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
  }
}

template <int D, int KV>
__global__ void __launch_bounds__(kThreads) read_tokens_kernel(const ReadParams p) {
  constexpr int E8 = D / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int per = p.hkv * E8;
  // (a 64-bit division only where the index needs it)
  const long long t = i <= 0xffffffffll ? static_cast<uint32_t>(i) / static_cast<uint32_t>(per) : i / per;
  const bool live = t < p.T;
  long long slot = -1;
  int bad = 0;
  if (live) {
    const int pos = p.positions[t];
    if (pos >= 0) {
      if (p.slots != nullptr) {
        const int s = p.slots[t];
        if (s < 0 || static_cast<long long>(s) >= static_cast<long long>(p.num_pages) * kPage) bad = LNK_DEV_BAD_SLOT;
        else slot = s;
      } else {
        const int row = p.rows != nullptr ? p.rows[t] : static_cast<int>(t);
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
  }
  // (the previous kernel on the stream may still write the pools or the status,
  // or read the outputs)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!live) return;
  const int rest = static_cast<int>(i - t * per);
  const int h = rest / E8, e8 = rest % E8;
  if (bad && rest == 0 && p.status != nullptr) atomicOr(p.status, bad);
  const size_t page = (static_cast<size_t>(h) * p.num_pages + static_cast<size_t>(slot / kPage)) * page_bytes(KV, D);
  uint4 v[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    v[which] = make_uint4(0u, 0u, 0u, 0u);
    if (slot >= 0 && p.out[which] != nullptr)
      v[which] = read8<D, KV>(p.pool[which] + page, static_cast<int>(slot % kPage), e8, p.scale[which]);
  }
#pragma unroll
  for (int which = 0; which < 2; ++which)
    if (p.out[which] != nullptr) reinterpret_cast<uint4*>(p.out[which])[i] = v[which];
}

template <int D, int KV>
cudaError_t launch_read_t(const ReadParams& p, cudaStream_t stream) {
  const long long n = static_cast<long long>(p.T) * p.hkv * (D / 8);
  const long long blocks = (n + kThreads - 1) / kThreads;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, read_tokens_kernel<D, KV>, p);
}

template <int D>
cudaError_t launch_read_d(const ReadParams& p, int kv_dtype, cudaStream_t stream) {
  switch (kv_dtype) {
    case LNK_KV_BF16: return launch_read_t<D, LNK_KV_BF16>(p, stream);
    case LNK_KV_E4M3: return launch_read_t<D, LNK_KV_E4M3>(p, stream);
    case LNK_KV_E2M1: return launch_read_t<D, LNK_KV_E2M1>(p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_read_tokens(const ReadParams& p, int head_dim, int kv_dtype, cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_read_d<64>(p, kv_dtype, stream);
    case 96: return launch_read_d<96>(p, kv_dtype, stream);
    case 128: return launch_read_d<128>(p, kv_dtype, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace lnk
