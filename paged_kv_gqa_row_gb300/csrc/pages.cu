// lnk_paged_copy_pages and lnk_paged_copy_pages_layers: copy whole pages of the
// K and V pools (every kv head) of one layer or of many, for the copy on write
// and the compaction of the host page allocator.
//
// A page of one head is contiguous (page_bytes); the unit of work is one such
// page of one pool: the grid is (kv heads * 2 pools * layers, page pairs), and
// a CTA moves its unit with 16-byte loads and stores, four of each in flight
// per thread.  The layers' pool addresses travel in the launch parameters, so
// a copy in every layer of a model is one launch and can be captured.  Bound by HBM:
// 160 pages of 8 heads in 32 layers, bf16 pools, D = 128, 2.7 GB read and written:
// 403 us, 6.6 TB/s; three pages: 8.9 us.
#include "common.cuh"
#include "latent.cuh"

namespace lnk {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kLayersPerLaunch = 128;

struct CopyParams {
  uint8_t* pool[2 * kLayersPerLaunch];  // layer l: K at 2 l, V at 2 l + 1
  const int32_t* src;
  const int32_t* dst;
  int32_t* status;
  int hkv, num_pages, units;  // units: 16-byte units per page of one head
  size_t head_stride, page_stride;  // 16-byte units from head to head and from page to page
  int first;                  // of the launch's page pairs
};

__global__ void __launch_bounds__(kThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  const int i = p.first + static_cast<int>(blockIdx.y);
  const int h = blockIdx.x % p.hkv, which = blockIdx.x / p.hkv;
  const int s = p.src[i], d = p.dst[i];
  if (s < 0 || s >= p.num_pages || d < 0 || d >= p.num_pages) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && p.status != nullptr) atomicOr(p.status, LNK_DEV_BAD_PAGE);
    return;
  }
  if (s == d) return;
  uint4* pool = reinterpret_cast<uint4*>(p.pool[which]);
  const uint4* from = pool + h * p.head_stride + s * p.page_stride;
  uint4* to = pool + h * p.head_stride + d * p.page_stride;
  for (int j = threadIdx.x; j < p.units; j += kUnroll * kThreads) {
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (j + u * kThreads < p.units) x[u] = __ldcs(from + j + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (j + u * kThreads < p.units) __stcs(to + j + u * kThreads, x[u]);
  }
}

lnk_status copy_pages(const lnk_attn_desc* desc, lnk_bf16* const* k_pools, lnk_bf16* const* v_pools, int32_t layers,
                      const int32_t* src_pages, const int32_t* dst_pages, int32_t n, int32_t* dev_status,
                      lnk_stream stream) {
  if (n == 0 || layers == 0) return LNK_OK;
  if (src_pages == nullptr || dst_pages == nullptr) return LNK_EINVAL;
  for (int32_t l = 0; l < layers; ++l)
    if (k_pools[l] == nullptr || v_pools[l] == nullptr) return LNK_EINVAL;
  if (desc->page_size != kPage) return LNK_EUNSUPPORTED;
  if (desc->head_dim != 64 && desc->head_dim != 96 && desc->head_dim != 128) return LNK_EUNSUPPORTED;
  if (desc->num_kv_heads <= 0 || desc->num_pages <= 0) return LNK_EINVAL;
  const int bytes = page_bytes(desc->kv_dtype, desc->head_dim);
  if (bytes == 0) return LNK_EUNSUPPORTED;
  for (int32_t l = 0; l < layers; ++l)
    if ((reinterpret_cast<uintptr_t>(k_pools[l]) | reinterpret_cast<uintptr_t>(v_pools[l])) % 16 != 0) return LNK_EINVAL;
  if (n > 65535 * 1024 || desc->num_kv_heads > 65535) return LNK_ERANGE;
  CopyParams p;
  p.src = src_pages;
  p.dst = dst_pages;
  p.status = dev_status;
  p.hkv = desc->num_kv_heads;
  p.num_pages = desc->num_pages;
  p.units = bytes / 16;
  p.page_stride = static_cast<size_t>(p.units);
  p.head_stride = static_cast<size_t>(p.num_pages) * p.units;
  for (int32_t l0 = 0; l0 < layers; l0 += kLayersPerLaunch) {
    const int32_t nl = layers - l0 < kLayersPerLaunch ? layers - l0 : kLayersPerLaunch;
    for (int32_t l = 0; l < nl; ++l) {
      p.pool[2 * l] = reinterpret_cast<uint8_t*>(k_pools[l0 + l]);
      p.pool[2 * l + 1] = reinterpret_cast<uint8_t*>(v_pools[l0 + l]);
    }
    for (int32_t i0 = 0; i0 < n; i0 += 65535) {
      p.first = i0;
      const dim3 grid(static_cast<unsigned>(p.hkv) * 2u * static_cast<unsigned>(nl),
                      static_cast<unsigned>(n - i0 < 65535 ? n - i0 : 65535));
      copy_pages_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
      if (cudaGetLastError() != cudaSuccess) return LNK_ECUDA;
    }
  }
  return LNK_OK;
}

}  // namespace
}  // namespace lnk

extern "C" lnk_status lnk_paged_copy_pages(const lnk_attn_desc* desc, lnk_bf16* k_pool, lnk_bf16* v_pool,
                                           const int32_t* src_pages, const int32_t* dst_pages, int32_t n,
                                           int32_t* dev_status, lnk_stream stream) {
  if (desc == nullptr || n < 0) return LNK_EINVAL;
  return lnk::copy_pages(desc, &k_pool, &v_pool, 1, src_pages, dst_pages, n, dev_status, stream);
}

extern "C" lnk_status lnk_paged_copy_pages_layers(const lnk_attn_desc* desc, lnk_bf16* const* k_pools,
                                                  lnk_bf16* const* v_pools, int32_t layers, const int32_t* src_pages,
                                                  const int32_t* dst_pages, int32_t n, int32_t* dev_status,
                                                  lnk_stream stream) {
  if (desc == nullptr || n < 0 || layers < 0) return LNK_EINVAL;
  if (layers > 0 && n > 0 && (k_pools == nullptr || v_pools == nullptr)) return LNK_EINVAL;
  return lnk::copy_pages(desc, k_pools, v_pools, layers, src_pages, dst_pages, n, dev_status, stream);
}

// A latent page is split into four parts, a CTA each, so that a copy of few pages spreads
// over the SMs (3 pages of 72 KB in 32 layers: 3.6 us, whole pages 5.6, halves 4.3; 160 pages in
// them, 755 MB: 112 us, whole pages 113.5).
extern "C" lnk_status lnk_latent_copy_pages(const lnk_latent_desc* desc, lnk_bf16* const* pools, int32_t layers,
                                            const int32_t* src_pages, const int32_t* dst_pages, int32_t n,
                                            int32_t* dev_status, lnk_stream stream) {
  using namespace lnk;
  const lnk_status st = check_latent_desc(desc);
  if (st != LNK_OK) return st;
  if (layers < 0 || n < 0) return LNK_EINVAL;
  if (layers == 0 || n == 0) return LNK_OK;
  if (pools == nullptr || src_pages == nullptr || dst_pages == nullptr) return LNK_EINVAL;
  for (int32_t l = 0; l < layers; ++l)
    if (pools[l] == nullptr || reinterpret_cast<uintptr_t>(pools[l]) % 16 != 0) return LNK_EINVAL;
  constexpr int kParts = 4;
  CopyParams p;
  p.src = src_pages;
  p.dst = dst_pages;
  p.status = dev_status;
  p.hkv = kParts;
  p.num_pages = desc->num_pages;
  p.units = kPage * (desc->latent_dim + desc->rope_dim) * 2 / 16 / kParts;
  p.head_stride = static_cast<size_t>(p.units);
  p.page_stride = static_cast<size_t>(p.units) * kParts;
  for (int32_t l0 = 0; l0 < layers; l0 += 2 * kLayersPerLaunch) {
    const int32_t nl = layers - l0 < 2 * kLayersPerLaunch ? layers - l0 : 2 * kLayersPerLaunch;
    for (int32_t l = 0; l < nl; ++l) p.pool[l] = reinterpret_cast<uint8_t*>(pools[l0 + l]);
    for (int32_t i0 = 0; i0 < n; i0 += 65535) {
      p.first = i0;
      const dim3 grid(static_cast<unsigned>(kParts * nl), static_cast<unsigned>(n - i0 < 65535 ? n - i0 : 65535));
      copy_pages_kernel<<<grid, kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
      if (cudaGetLastError() != cudaSuccess) return LNK_ECUDA;
    }
  }
  return LNK_OK;
}
