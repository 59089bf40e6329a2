// Parameter blocks and launchers of the latent-cache kernels.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace lnk {

constexpr int kLatentRows = 64;  // query rows of a one-SM attention tile at most
constexpr int kWholePages = 8;   // tokens of so few pages are never cut

// A softmax reference (log2 units) is set this far above a score, and raised when another score
// exceeds it by the second.
constexpr float kAheadLog2 = 24.f;
constexpr float kRaiseLog2 = 8.f;

// Rows that attend_again computes again can take longer than a wait may: their
// warps keep writing the time into the beat, a word of each CTA of the cluster from which the
// other roles' limits count.  It lies kBeat words behind the abort flag.
constexpr int kBeat = 3;
template <bool kPair>
__device__ __forceinline__ void beat(volatile int* abort) {
  if ((threadIdx.x & 31) != 0) return;
  const int now = static_cast<int>(beat_now());
  abort[kBeat] = now;
  if (kPair) st_shared_remote(mapa_shared(smem_addr(const_cast<int*>(abort) + kBeat), cluster_cta_rank() ^ 1u), now);
}

__device__ __forceinline__ bool wait_with_beat(uint32_t bar, uint32_t parity, volatile int* abort) {
  return mbar_wait(bar, parity, abort, kWaitLimitNs, abort + kBeat);
}

__device__ __forceinline__ float bf16_at(const uint16_t* x) {
  return __uint_as_float(static_cast<uint32_t>(*x) << 16);
}

// Bits 15 and 31: a bf16 number among eight is not finite.
__device__ __forceinline__ uint32_t odd_halves(const uint4& x) {
  auto odd = [](uint32_t w) { return (w & 0x7F807F80u) + 0x00800080u; };
  return (odd(x.x) | odd(x.y) | odd(x.z) | odd(x.w)) & 0x80008000u;
}

// s + the products of eight pairs of bf16 numbers
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b, float s) {
  auto two = [&s](uint32_t x, uint32_t y) {
    s = fmaf(__uint_as_float(x << 16), __uint_as_float(y << 16), s);
    s = fmaf(__uint_as_float(x & 0xFFFF0000u), __uint_as_float(y & 0xFFFF0000u), s);
  };
  two(a.x, b.x);
  two(a.y, b.y);
  two(a.z, b.z);
  two(a.w, b.w);
  return s;
}

// A row of a tile (a unit of the stream of pages) that the teams' shares cut: what
// the joining kernel needs to know, written by the team whose share starts inside it.
struct LatentCut {
  int32_t t0, nt;     // the unit's first token and its tokens
  int32_t j0;         // pages of the unit before the share (0: the share starts with a unit)
  int32_t np;         // pages of the unit
  long long per;      // pages of a share
  long long pad;
};

struct LatentParams {
  const uint16_t* q;               // [T][H][C + R]
  const uint16_t* pool;            // [num_pages * 64][C + R]
  const int32_t* rows;             // [P]
  const int32_t* positions;        // [P]
  const int32_t* step_positions;   // [T - P]
  const int32_t* table;
  uint16_t* out;                   // [T][H][C]
  int32_t* status;
  LatentCut* cuts;                 // [teams]
  float* ml;                       // [2 * teams * head blocks][slot rows][2]: reference (log2 units), sum
  float* o;                        // [2 * teams * head blocks][slot rows][C]: unnormalised partial outputs
  int P, T, heads, latent_dim, rope_dim, num_pages, num_rows, pages_per_row, window;
  int tile_rows;                   // query rows a tile (128: on pairs of SMs; 64, 32 or 16)
  int slot_rows;                   // rows of a partial sum in the workspace
  int tile_tokens;                 // prompt tokens a tile at most
  int head_blocks;                 // tiles a token (heads > tile_rows)
  int teams;                       // groups of head_blocks CTAs (or pairs) that share the stream
  int whole;                       // no unit is cut (all have few pages)
  float scale_log2;
};

// qmap: query rows; pmap: the pool as [8 keys][64 numbers][row of 8][number of 64], boxes of 16
// keys, or of 8 and without the rotated part where that has 32 numbers; rmap: that part.
cudaError_t launch_latent_attn(const CUtensorMap& qmap, const CUtensorMap& pmap, const CUtensorMap& rmap,
                               const LatentParams& p, cudaStream_t stream);

// The same with tiles of 128 rows on pairs of SMs.  qmap: boxes of 64 rows; kmap: the pool as
// [8 keys][64 numbers] blocks, boxes of 32 keys (with a rotated part of 32: of 8 keys, without
// it, and rmap that part); vmap: boxes of 64 keys and half of a latent.
cudaError_t launch_latent_pair(const CUtensorMap& qmap, const CUtensorMap& kmap, const CUtensorMap& vmap,
                               const CUtensorMap& rmap, const LatentParams& p, cudaStream_t stream);

// Joins the partial sums that either of them left.
cudaError_t launch_latent_join(const LatentParams& p, cudaStream_t stream);

struct LatentAppendParams {
  const uint16_t* q;        // [T][H] rotated parts, q_stride elements from head to head
  const uint16_t* kv;       // [T][C + R]
  const int32_t* positions;
  const int32_t* rows;
  const int32_t* slots;
  const int32_t* table;
  const uint16_t* norm_w;   // [C] or null
  uint16_t* pool;
  uint16_t* q_out;
  uint16_t* kv_out;         // or null
  int32_t* status;
  double norm_eps;
  float inv_dim[2], eps[2];  // 1 / C and the epsilon as float pairs
  long long q_stride, q_out_stride;
  int T, heads, latent_dim, rope_dim, num_pages, num_rows, pages_per_row;
  float inv_freq[32];
};

cudaError_t launch_latent_append(const LatentAppendParams& p, cudaStream_t stream);

struct LatentPromptParams {
  const uint16_t* q;         // [Tq][H][D + R]
  const uint16_t* kv;        // [Tk][H][2 D]
  const uint16_t* k_rope;    // [Tk], rope_stride elements from token to token
  const int32_t* q_starts;   // [prompts + 1]
  const int32_t* k_starts;
  uint16_t* out;             // [Tq][H][D]
  int32_t* status;
  long long rope_stride;
  int heads, head_dim, rope_dim, Tq, Tk, prompts;
  int tiles;                 // ids of tiles
  float scale_log2;
};

int latent_prompt_tile_rows();
cudaError_t launch_latent_prompt(const CUtensorMap& qmap, const CUtensorMap& kvmap, const CUtensorMap& rmap,
                                 const LatentPromptParams& p, cudaStream_t stream);

lnk_status check_latent_desc(const lnk_latent_desc* desc);

// A tensor map over bf16 data of 2 to 4 dimensions (sizes and, from the second on,
// strides in elements), boxes of `box` elements, 128-byte swizzle.
bool bf16_tensor_map(CUtensorMap* map, const void* base, int rank, const long long* dims, const long long* strides,
                     const int* box);

// The float32 frequencies of a rotation of `dim` elements (lnk_rope_inv_freq).
lnk_status rope_frequencies(const lnk_rope_desc* rope, int dim, float* out);

}  // namespace lnk
