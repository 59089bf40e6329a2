// C entry points of the latent cache: argument checks and launches.
#include <algorithm>
#include <cfloat>
#include <cstring>

#include "latent.cuh"

namespace lnk {
namespace {

constexpr int kMaxLatentHeads = 1024;

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

float latent_scale_log2(const lnk_latent_desc* d) {
  return static_cast<float>(static_cast<double>(d->scale) * 1.4426950408889634);  // log2(e)
}

lnk_status check_desc(const lnk_latent_desc* d) {
  if (d == nullptr) return LNK_EINVAL;
  if (d->page_size != kPage) return LNK_EUNSUPPORTED;
  if (d->latent_dim != 128 && d->latent_dim != 256 && d->latent_dim != 384 && d->latent_dim != 512)
    return LNK_EUNSUPPORTED;
  if (d->rope_dim != 32 && d->rope_dim != 64) return LNK_EUNSUPPORTED;
  if (d->num_heads <= 0) return LNK_EINVAL;
  if (d->num_heads > kMaxLatentHeads) return LNK_ERANGE;
  if (d->num_pages <= 0 || d->num_rows <= 0 || d->pages_per_row <= 0) return LNK_EINVAL;
  if (d->window < 0 || !(d->scale > 0.f)) return LNK_EINVAL;
  // (a zero or infinite factor would make NaN of masked scores and of zero ones)
  if (!(latent_scale_log2(d) > 0.f && latent_scale_log2(d) <= FLT_MAX)) return LNK_ERANGE;
  // TMA row coordinates and 32-bit position arithmetic must not overflow
  if (static_cast<long long>(d->num_pages) * kPage >= (1ll << 31)) return LNK_ERANGE;
  if (static_cast<long long>(d->pages_per_row) * kPage >= (1ll << 31)) return LNK_ERANGE;
  if (static_cast<long long>(d->num_rows) * d->pages_per_row >= (1ll << 31)) return LNK_ERANGE;
  return LNK_OK;
}

struct Workspace {
  size_t cuts, ml, o, total;
};

// The partial sums of two cut units a CTA, each of kLatentRows rows at most.
Workspace workspace_layout(int ctas, int latent_dim) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  Workspace w;
  w.cuts = 0;
  w.ml = up(sizeof(LatentCut) * static_cast<size_t>(ctas));
  w.o = w.ml + up(sizeof(float) * 2 * 2 * static_cast<size_t>(ctas) * kLatentRows);
  w.total = w.o + sizeof(float) * 2 * static_cast<size_t>(ctas) * kLatentRows * static_cast<size_t>(latent_dim);
  return w;
}

lnk_status attend(const lnk_latent_desc* desc, const lnk_bf16* q, const int32_t* rows, const int32_t* positions,
                  const int32_t* step_positions, const int32_t* table, const lnk_bf16* pool, lnk_bf16* out, int32_t P,
                  int32_t B, void* workspace, size_t ws_bytes, int32_t* dev_status, lnk_stream stream) {
  const lnk_status st = check_desc(desc);
  if (st != LNK_OK) return st;
  if (P < 0 || B < 0 || B > desc->num_rows) return LNK_EINVAL;
  if (B > kMaxDecodeRows) return LNK_ERANGE;
  if ((static_cast<long long>(P) + B) * desc->num_heads >= (1ll << 31)) return LNK_ERANGE;
  if (P == 0 && B == 0) return LNK_OK;
  if (!q || !table || !pool || !out) return LNK_EINVAL;
  if (P > 0 && (!rows || !positions)) return LNK_EINVAL;
  if (B > 0 && !step_positions) return LNK_EINVAL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(pool, 16)) return LNK_EINVAL;
  const int sms = device_sm_count();
  if (sms <= 0) return LNK_ECUDA;
  const Workspace w = workspace_layout(sms, desc->latent_dim);
  if (workspace == nullptr || ws_bytes < w.total || !aligned(workspace, 256)) return LNK_EWORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  LatentParams p;
  std::memset(&p, 0, sizeof(p));
  p.q = q;
  p.pool = pool;
  p.rows = rows;
  p.positions = positions;
  p.step_positions = step_positions;
  p.table = table;
  p.out = out;
  p.status = dev_status;
  p.cuts = reinterpret_cast<LatentCut*>(ws + w.cuts);
  p.ml = reinterpret_cast<float*>(ws + w.ml);
  p.o = reinterpret_cast<float*>(ws + w.o);
  p.P = P;
  p.T = P + B;
  p.heads = desc->num_heads;
  p.latent_dim = desc->latent_dim;
  p.rope_dim = desc->rope_dim;
  p.num_pages = desc->num_pages;
  p.num_rows = desc->num_rows;
  p.pages_per_row = desc->pages_per_row;
  p.window = desc->window;
  // Tiles of 128 rows on pairs of SMs for more heads than 64 (64 decode rows of 128 heads: 85.6
  // us so, 111 in two tiles of 64), and for launches of so many prompt tokens that their
  // products weigh more than the pages' way to the SMs (with 32 decode rows of 2000 to 4000 keys,
  // 4 pieces of 32 tokens of 64 heads: 88 us so, 110 in tiles of 64; of 16 tokens 66 and 70; of 4
  // 49 and 49; of 16 tokens of 16 heads 49 and 47).  Else tiles of 64, or of 32 or 16 for decode
  // rows of fewer heads, which never share a tile (64 rows of 16 heads, 3000 to 5000 keys: 59.8
  // us in 16, 61.4 in 32, 66.4 in 64, 74.1 on pairs).
  const bool pairs = p.heads > kLatentRows || static_cast<long long>(P) * p.heads >= static_cast<long long>(sms) * 16;
  p.tile_rows = pairs ? 2 * kLatentRows : (P > 0 || p.heads > 32 ? 64 : (p.heads > 16 ? 32 : 16));
  p.slot_rows = std::max(kLatentRows, p.tile_rows);
  p.tile_tokens = std::max(1, p.tile_rows / p.heads);
  p.head_blocks = (p.heads + p.tile_rows - 1) / p.tile_rows;
  p.teams = (pairs ? sms / 2 : sms) / p.head_blocks;
  if (p.teams <= 0) return LNK_ERANGE;
  long long most = p.pages_per_row;  // pages of a token
  if (p.window > 0) most = std::min<long long>(most, (p.window - 1) / kPage + 2);
  p.whole = most <= kWholePages;  // (and there is no second kernel: 64 rows of 100 to 500 keys 17.4 us so, 19.6 with it)
  p.scale_log2 = latent_scale_log2(desc);

  const long long width = desc->latent_dim + desc->rope_dim;
  const long long qdims[2] = {width, static_cast<long long>(p.T) * p.heads};
  const long long keys8 = static_cast<long long>(p.num_pages) * kPage / 8;
  const long long pdims[4] = {kBoxCols, 8, width / kBoxCols, keys8};
  const long long rdims[2] = {width, static_cast<long long>(p.num_pages) * kPage};
  const long long strides[2] = {1, width}, pstrides[4] = {1, width, kBoxCols, 8 * width};
  // with a rotated part of 32 numbers a row is no multiple of 64: that part has copies of its own
  const bool r64 = p.rope_dim == 64;
  const int qbox[2] = {kBoxCols, std::min(p.tile_rows, kLatentRows)}, rbox[2] = {kBoxCols, 8};
  const int pbox[4] = {kBoxCols, 8, static_cast<int>(width / kBoxCols), r64 ? (pairs ? 4 : 2) : 1};
  const int vbox[4] = {kBoxCols, 8, p.latent_dim / 2 / kBoxCols, 8};
  CUtensorMap qmap, pmap, vmap, rmap;
  if (!bf16_tensor_map(&qmap, q, 2, qdims, strides, qbox) || !bf16_tensor_map(&pmap, pool, 4, pdims, pstrides, pbox))
    return LNK_ECUDA;
  if (r64) rmap = pmap;  // (not used)
  else if (!bf16_tensor_map(&rmap, pool, 2, rdims, strides, rbox)) return LNK_ECUDA;
  if (pairs && !bf16_tensor_map(&vmap, pool, 4, pdims, pstrides, vbox)) return LNK_ECUDA;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t err = pairs ? launch_latent_pair(qmap, pmap, vmap, rmap, p, s) : launch_latent_attn(qmap, pmap, rmap, p, s);
  return err == cudaSuccess ? LNK_OK : LNK_ECUDA;
}

}  // namespace

lnk_status check_latent_desc(const lnk_latent_desc* desc) { return check_desc(desc); }

}  // namespace lnk

using namespace lnk;

extern "C" {

size_t lnk_latent_workspace_size(const lnk_latent_desc* desc) {
  if (check_desc(desc) != LNK_OK) return 0;
  const int sms = device_sm_count();
  return sms > 0 ? workspace_layout(sms, desc->latent_dim).total : 0;
}

lnk_status lnk_latent_append(const lnk_latent_desc* desc, const lnk_rope_desc* rope, const lnk_bf16* q,
                             int64_t q_stride, const lnk_bf16* kv, const int32_t* positions, const int32_t* rows,
                             const int32_t* slots, const int32_t* table, const lnk_bf16* norm_w, float norm_eps,
                             lnk_bf16* pool, lnk_bf16* q_out, int64_t q_out_stride, lnk_bf16* kv_out, int32_t T,
                             int32_t* dev_status, lnk_stream stream) {
  lnk_status st = check_desc(desc);
  if (st != LNK_OK) return st;
  if (T < 0) return LNK_EINVAL;
  if (T == 0) return LNK_OK;
  if (!q || !kv || !positions || !pool || !q_out || (!slots && !table)) return LNK_EINVAL;
  if (!aligned(q, 4) || !aligned(q_out, 4) || !aligned(kv, 16) || !aligned(pool, 16) || !aligned(kv_out, 16) ||
      !aligned(norm_w, 16))
    return LNK_EINVAL;
  if (q_stride < desc->rope_dim || q_out_stride < desc->rope_dim || q_stride % 2 != 0 || q_out_stride % 2 != 0)
    return LNK_EINVAL;
  // (byte offsets of the last token must stay within 63 bits)
  if (q_stride > (1ll << 30) || q_out_stride > (1ll << 30)) return LNK_ERANGE;
  if (norm_w && !(norm_eps >= 0.f)) return LNK_EINVAL;
  if (rows == nullptr && slots == nullptr && T > desc->num_rows) return LNK_EINVAL;
  LatentAppendParams p;
  std::memset(&p, 0, sizeof(p));
  st = rope_frequencies(rope, desc->rope_dim, p.inv_freq);
  if (st != LNK_OK) return st;
  p.q = q;
  p.kv = kv;
  p.positions = positions;
  p.rows = rows;
  p.slots = slots;
  p.table = table;
  p.norm_w = norm_w;
  p.pool = pool;
  p.q_out = q_out;
  p.kv_out = kv_out;
  p.status = dev_status;
  p.norm_eps = static_cast<double>(norm_eps);
  const double inv_dim = 1.0 / desc->latent_dim;
  p.inv_dim[0] = static_cast<float>(inv_dim);
  p.inv_dim[1] = static_cast<float>(inv_dim - static_cast<double>(p.inv_dim[0]));
  p.eps[0] = norm_eps;
  p.q_stride = q_stride;
  p.q_out_stride = q_out_stride;
  p.T = T;
  p.heads = desc->num_heads;
  p.latent_dim = desc->latent_dim;
  p.rope_dim = desc->rope_dim;
  p.num_pages = desc->num_pages;
  p.num_rows = desc->num_rows;
  p.pages_per_row = desc->pages_per_row;
  return launch_latent_append(p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LNK_OK : LNK_ECUDA;
}

lnk_status lnk_latent_decode_attn(const lnk_latent_desc* desc, const lnk_bf16* q, const int32_t* positions,
                                  const int32_t* table, const lnk_bf16* pool, lnk_bf16* out, int32_t B, void* workspace,
                                  size_t ws_bytes, int32_t* dev_status, lnk_stream stream) {
  return attend(desc, q, nullptr, nullptr, positions, table, pool, out, 0, B, workspace, ws_bytes, dev_status, stream);
}

lnk_status lnk_latent_step_attn(const lnk_latent_desc* desc, const lnk_bf16* q, const int32_t* rows,
                                const int32_t* positions, const int32_t* step_positions, const int32_t* table,
                                const lnk_bf16* pool, lnk_bf16* out, int32_t P, int32_t B, void* workspace,
                                size_t ws_bytes, int32_t* dev_status, lnk_stream stream) {
  return attend(desc, q, rows, positions, step_positions, table, pool, out, P, B, workspace, ws_bytes, dev_status,
                stream);
}

lnk_status lnk_latent_prompt_attn(int32_t num_heads, int32_t head_dim, int32_t rope_dim, float scale, const lnk_bf16* q,
                                  const lnk_bf16* kv, const lnk_bf16* k_rope, int64_t k_rope_stride,
                                  const int32_t* q_starts, const int32_t* k_starts, lnk_bf16* out, int32_t Tq, int32_t Tk,
                                  int32_t N, int32_t* dev_status, lnk_stream stream) {
  if (num_heads <= 0 || Tq < 0 || Tk < 0 || N < 0 || !(scale > 0.f)) return LNK_EINVAL;
  if ((head_dim != 64 && head_dim != 128) || (rope_dim != 32 && rope_dim != 64)) return LNK_EUNSUPPORTED;
  if (num_heads > kMaxLatentHeads) return LNK_ERANGE;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // log2(e)
  if (!(scale_log2 > 0.f && scale_log2 <= FLT_MAX)) return LNK_ERANGE;
  if (Tq == 0 || N == 0) return LNK_OK;
  if (!q || !q_starts || !k_starts || !out) return LNK_EINVAL;
  if (Tk > 0 && (!kv || !k_rope)) return LNK_EINVAL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(k_rope, 16) || !aligned(out, 16)) return LNK_EINVAL;
  if (k_rope_stride < rope_dim || k_rope_stride % 8 != 0) return LNK_EINVAL;
  if (k_rope_stride > (1ll << 30)) return LNK_ERANGE;
  if (Tk == 0) {  // no prompt has a key: every query's output is zero (of the queries that a prompt holds)
    kv = q;
    k_rope = q;
  }
  const int rows = latent_prompt_tile_rows();
  LatentPromptParams p;
  p.q = q;
  p.kv = kv;
  p.k_rope = k_rope;
  p.q_starts = q_starts;
  p.k_starts = k_starts;
  p.out = out;
  p.status = dev_status;
  p.rope_stride = k_rope_stride;
  p.heads = num_heads;
  p.head_dim = head_dim;
  p.rope_dim = rope_dim;
  p.Tq = Tq;
  p.Tk = Tk;
  p.prompts = N;
  const long long tiles = static_cast<long long>(Tq) / rows + N;
  if (2 * tiles * num_heads > 0x7fffffffll) return LNK_ERANGE;
  p.tiles = static_cast<int>(tiles);
  p.scale_log2 = scale_log2;
  const long long h = num_heads, tk = std::max(1, Tk);
  const long long qdims[3] = {head_dim + rope_dim, h, Tq}, qstr[3] = {1, head_dim + rope_dim, h * (head_dim + rope_dim)};
  const long long kdims[3] = {2 * head_dim, h, tk}, kstr[3] = {1, 2 * head_dim, h * 2 * head_dim};
  const long long rdims[2] = {rope_dim, tk}, rstr[2] = {1, k_rope_stride};
  const int qbox[3] = {kBoxCols, 1, rows / 2}, kbox[3] = {kBoxCols, 1, 64}, rbox[2] = {kBoxCols, 64};
  CUtensorMap qmap, kvmap, rmap;
  if (!bf16_tensor_map(&qmap, q, 3, qdims, qstr, qbox) || !bf16_tensor_map(&kvmap, kv, 3, kdims, kstr, kbox) ||
      !bf16_tensor_map(&rmap, k_rope, 2, rdims, rstr, rbox))
    return LNK_ECUDA;
  return launch_latent_prompt(qmap, kvmap, rmap, p, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? LNK_OK
                                                                                                          : LNK_ECUDA;
}

}  // extern "C"
