// C ABI of libnvfp4.so (declared in include/nvfp4.h): argument validation,
// kernel choice and error reporting.  Every check runs on the host before
// any HIP call, so a rejected call enqueues nothing and touches no device.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/nvfp4.h"
#include "kv_cache.h"
#include "launch.h"

namespace {

thread_local char g_last_error[512] = "";

nvfp4_status fail(nvfp4_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
  va_end(ap);
  return s;
}

nvfp4_status ok() {
  g_last_error[0] = '\0';
  return NVFP4_OK;
}

nvfp4_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(NVFP4_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
  const void* p;
  int64_t bytes;
  const char* name;
};

bool overlap(const Range& a, const Range& b) {
  if (a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + (uintptr_t)b.bytes && b0 < a0 + (uintptr_t)a.bytes;
}

// Checks that no output range overlaps any other listed range.
nvfp4_status check_disjoint(const Range* outs, int nout, const Range* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlap(outs[i], ins[j]))
        return fail(NVFP4_ERR_INVALID_ARG, "output %s overlaps input %s", outs[i].name, ins[j].name);
    for (int j = i + 1; j < nout; ++j)
      if (overlap(outs[i], outs[j]))
        return fail(NVFP4_ERR_INVALID_ARG, "output %s overlaps output %s", outs[i].name, outs[j].name);
  }
  return NVFP4_OK;
}

constexpr int64_t kMaxDim = 0x7FFFFFFF;
// The INT4 and weight-only NVFP4 tiled kernels address a tile's rows of x
// (128 x 2K bytes) with 32-bit buffer offsets.
constexpr int64_t kInt4TiledKLimit = (int64_t)1 << 22;
// The weight-streaming kernels address at most kDecodeMaxRows packed weight
// rows (the 112-row workgroup of the INT4 decode kernel is the largest) and
// the whole bf16 activation of M <= 16 rows through buffer resources with
// 32-bit byte ranges.  Offsets at or past 2^31 mark loads that must read
// zero, so every range must stay below 2^31; K <= 2^24 guarantees it.
constexpr int64_t kDecodeMaxK = int64_t(1) << 24;
constexpr int64_t kDecodeMaxRows = 112;
constexpr int64_t kBufferOobOffset = int64_t(1) << 31;
static_assert(kDecodeMaxRows * (kDecodeMaxK / 2) < kBufferOobOffset, "weight rows of a decode workgroup");
static_assert(16 * kDecodeMaxK * 2 < kBufferOobOffset, "bf16 activation of a decode call");
// The NVFP4 tiled kernel addresses a tile's rows (256 x K/2 bytes) with
// 32-bit buffer offsets.
constexpr int64_t kTiledKLimit = int64_t(1) << 24;

#define REQUIRE_PTR(p)                                                               \
  do {                                                                               \
    if ((p) == nullptr) return fail(NVFP4_ERR_INVALID_ARG, "%s is a null pointer", #p); \
  } while (0)
#define REQUIRE_ALIGN(p, a)                                                                  \
  do {                                                                                       \
    if (!aligned((p), (a))) return fail(NVFP4_ERR_ALIGNMENT, "%s is not %d-byte aligned", #p, (int)(a)); \
  } while (0)

nvfp4_status check_dims(int64_t a, const char* an, int64_t b, const char* bn, int64_t c, const char* cn) {
  if (a < 0 || b < 0 || c < 0)
    return fail(NVFP4_ERR_INVALID_ARG, "negative size (%s=%lld, %s=%lld, %s=%lld)", an, (long long)a, bn,
                (long long)b, cn, (long long)c);
  if (a > kMaxDim || b > kMaxDim || c > kMaxDim)
    return fail(NVFP4_ERR_UNSUPPORTED, "a dimension exceeds 2^31-1 (%s=%lld, %s=%lld, %s=%lld)", an,
                (long long)a, bn, (long long)b, cn, (long long)c);
  return NVFP4_OK;
}

// Matrix sizes whose element counts stay below 2^40 (far past any device
// memory), so byte counts and ranges never overflow int64.
constexpr int64_t kMaxElems = int64_t(1) << 40;
nvfp4_status check_products(int64_t M, int64_t N, int64_t K) {
  if ((N > 0 && M > kMaxElems / N) || (K > 0 && M > kMaxElems / K) || (K > 0 && N > kMaxElems / K))
    return fail(NVFP4_ERR_UNSUPPORTED, "a matrix exceeds 2^40 elements (M=%lld, N=%lld, K=%lld)", (long long)M,
                (long long)N, (long long)K);
  return NVFP4_OK;
}

// Which kernel AUTO picks for the NVFP4 GEMM.
int auto_algo(int64_t M, int64_t K) {
  const bool k128 = (K % 128) == 0 && K > 0;
  return !k128 ? NVFP4_ALGO_SIMPLE
               : (M <= 16 ? (K <= kDecodeMaxK ? NVFP4_ALGO_DECODE : NVFP4_ALGO_SIMPLE)
                          : (K < kTiledKLimit ? NVFP4_ALGO_TILED : NVFP4_ALGO_SIMPLE));
}

// Slots nvfp4_gemm_amax writes for AUTO's kernel choice: one per output tile
// of the tiled kernel, else the partial maxima of a separate pass over out.
int64_t amax_slots(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0) return 0;
  if (auto_algo(M, K) == NVFP4_ALGO_TILED) return nvfp4k::nvfp4_gemm_tiled_amax_slots(M, N);
  return nvfp4k::amax_partial_count(M * N);
}

// Shared by nvfp4_gemm_ex, nvfp4_gemm_lora_ex and nvfp4_gemm_amax; lora_t ==
// nullptr means no low-rank branch (its arguments were validated by the
// caller); amax != nullptr (AUTO, no branch, N % 16 == 0) also writes the
// output's amax slots.
nvfp4_status gemm_impl(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                       const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale, void* out_bf16,
                       int64_t M, int64_t N, int64_t K, int algo, const float* lora_t, const void* lora_up,
                       int64_t r, void* workspace, size_t workspace_bytes, void* stream, uint32_t* amax = nullptr) {
  if (nvfp4_status s = check_dims(M, "M", N, "N", K, "K")) return s;
  if (nvfp4_status s = check_products(M, N, K)) return s;
  if (K > 0) {  // with K == 0 the packed operands are empty and never read
    REQUIRE_PTR(a_codes);
    REQUIRE_PTR(a_scales);
    REQUIRE_PTR(w_codes);
    REQUIRE_PTR(w_scales);
  }
  REQUIRE_PTR(a_gscale);
  REQUIRE_PTR(w_gscale);
  REQUIRE_PTR(out_bf16);
  if (K % 16 != 0) return fail(NVFP4_ERR_SHAPE, "K=%lld is not a multiple of 16", (long long)K);
  if (algo < NVFP4_ALGO_AUTO || algo > NVFP4_ALGO_SIMPLE) return fail(NVFP4_ERR_INVALID_ARG, "unknown algo %d", algo);
  REQUIRE_ALIGN(a_codes, 16);
  REQUIRE_ALIGN(a_scales, 16);
  REQUIRE_ALIGN(w_codes, 16);
  REQUIRE_ALIGN(w_scales, 16);
  REQUIRE_ALIGN(out_bf16, 16);
  REQUIRE_ALIGN(a_gscale, 4);
  REQUIRE_ALIGN(w_gscale, 4);
  if (workspace != nullptr) {
    REQUIRE_ALIGN(workspace, 256);
    if (workspace_bytes > (size_t)INT64_MAX) return fail(NVFP4_ERR_INVALID_ARG, "workspace_bytes is too large");
  }
  const Range outs[3] = {{out_bf16, M * N * 2, "out"},
                         {workspace, workspace ? (int64_t)workspace_bytes : 0, "workspace"},
                         {amax, amax ? 4 * amax_slots(M, N, K) : 0, "amax_slots"}};
  const Range ins[8] = {{a_codes, M * K / 2, "a_codes"}, {a_scales, M * K / 16, "a_scales"},
                        {a_gscale, 4, "a_gscale"},       {w_codes, N * K / 2, "w_codes"},
                        {w_scales, N * K / 16, "w_scales"}, {w_gscale, 4, "w_gscale"},
                        {lora_t, lora_t ? M * r * 4 : 0, "lora_t"}, {lora_up, lora_t ? N * r * 2 : 0, "lora_up"}};
  if (M == 0 || N == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 3, ins, 8)) return s;
  const bool k128 = (K % 128) == 0 && K > 0;
  if (algo == NVFP4_ALGO_AUTO) algo = auto_algo(M, K);
  hipStream_t st = (hipStream_t)stream;
  if (amax && algo != NVFP4_ALGO_TILED) {    // the output's maxima from a separate pass
    nvfp4_status s = gemm_impl(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K, algo,
                               nullptr, nullptr, 0, workspace, workspace_bytes, stream);
    if (s != NVFP4_OK) return s;
    return hip_status(nvfp4k::launch_amax_partials(out_bf16, M * N, amax, st), "nvfp4_gemm_amax amax pass");
  }
  switch (algo) {
    case NVFP4_ALGO_TILED:
      if (!k128 || K >= kTiledKLimit)
        return fail(NVFP4_ERR_UNSUPPORTED, "tiled kernel needs K %% 128 == 0 and 0 < K < 2^24 (K=%lld)", (long long)K);
      if (lora_t)
        return hip_status(nvfp4k::launch_nvfp4_gemm_tiled_lora(a_codes, a_scales, a_gscale, w_codes, w_scales,
                                                               w_gscale, out_bf16, M, N, K, lora_t, lora_up, r, st),
                          "nvfp4_gemm_lora tiled launch");
      return hip_status(nvfp4k::launch_nvfp4_gemm_tiled_ws(a_codes, a_scales, a_gscale, w_codes, w_scales,
                                                           w_gscale, out_bf16, M, N, K, workspace,
                                                           (int64_t)workspace_bytes, st, amax),
                        "nvfp4_gemm tiled launch");
    case NVFP4_ALGO_DECODE:
      if (!k128 || M > 16 || K > kDecodeMaxK)
        return fail(NVFP4_ERR_UNSUPPORTED, "decode kernel needs M <= 16, K %% 128 == 0 and K <= 2^24 (M=%lld, K=%lld)",
                    (long long)M, (long long)K);
      return hip_status(nvfp4k::launch_nvfp4_gemm_decode_lora(a_codes, a_scales, a_gscale, w_codes, w_scales,
                                                              w_gscale, out_bf16, M, N, K, lora_t, lora_up, r, st),
                        "nvfp4_gemm decode launch");
    default:
      return hip_status(nvfp4k::launch_nvfp4_gemm_simple_lora(a_codes, a_scales, a_gscale, w_codes, w_scales,
                                                              w_gscale, out_bf16, M, N, K, lora_t, lora_up, r, st),
                        "nvfp4_gemm simple launch");
  }
}

// Rank limits shared by the two low-rank entry points.
nvfp4_status check_rank(int64_t r) {
  if (r < 8 || r > nvfp4k::kLoraMaxRank || r % 8 != 0)
    return fail(NVFP4_ERR_UNSUPPORTED, "rank r=%lld; supported ranks are multiples of 8 in [8, %d]", (long long)r,
                nvfp4k::kLoraMaxRank);
  return NVFP4_OK;
}

// ---- NVFP4 key/value cache ----

// A strided [tokens][width] matrix (stride and width in bytes) as a range.
int64_t strided_bytes(int64_t tokens, int64_t stride, int64_t width) {
  return tokens > 0 ? (tokens - 1) * stride + width : 0;
}

// Whether two strided matrices share a byte.  Views of one buffer with the
// same stride (q and k in a packed QKV row) interleave without sharing any.
bool strided_overlap(const void* a, int64_t a_stride, int64_t a_width, const void* b, int64_t b_stride,
                     int64_t b_width, int64_t tokens) {
  const Range ra{a, strided_bytes(tokens, a_stride, a_width), ""}, rb{b, strided_bytes(tokens, b_stride, b_width), ""};
  if (!overlap(ra, rb)) return false;
  if (a_stride != b_stride || a_stride <= 0) return true;
  const int64_t diff = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t off = ((diff % a_stride) + a_stride) % a_stride;
  return !(off >= a_width && off + b_width <= a_stride);
}

nvfp4_status check_cache(const nvfp4_kv_cache* c, nvfp4k::KvCache* out) {
  if (c == nullptr) return fail(NVFP4_ERR_INVALID_ARG, "cache is a null pointer");
  if (nvfp4_status s = check_dims(c->num_pages, "num_pages", c->page_size, "page_size", c->kv_heads, "kv_heads"))
    return s;
  if (c->page_size < 16 || c->page_size > 4096 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(NVFP4_ERR_SHAPE, "page_size=%lld is not a power of two in [16, 4096]", (long long)c->page_size);
  if (c->kv_heads < 1 || c->kv_heads > 65535)
    return fail(NVFP4_ERR_UNSUPPORTED, "kv_heads=%lld; 1 to 65535 are supported", (long long)c->kv_heads);
  if (!nvfp4k::kv_head_dim_supported(c->head_dim))
    return fail(NVFP4_ERR_UNSUPPORTED, "head_dim=%lld; supported head sizes are 64, 128 and 256",
                (long long)c->head_dim);
  if (c->num_pages > kMaxElems / (c->page_size * c->kv_heads * c->head_dim))
    return fail(NVFP4_ERR_UNSUPPORTED, "the cache exceeds 2^40 elements");
  if (c->num_pages > 0) {
    REQUIRE_PTR(c->k_codes);
    REQUIRE_PTR(c->k_scales);
    REQUIRE_PTR(c->v_codes);
    REQUIRE_PTR(c->v_scales);
  }
  REQUIRE_PTR(c->k_gscale);
  REQUIRE_PTR(c->v_gscale);
  REQUIRE_ALIGN(c->k_codes, 16);
  REQUIRE_ALIGN(c->k_scales, 16);
  REQUIRE_ALIGN(c->v_codes, 16);
  REQUIRE_ALIGN(c->v_scales, 16);
  REQUIRE_ALIGN(c->k_gscale, 4);
  REQUIRE_ALIGN(c->v_gscale, 4);
  int lg = 0;
  while ((int64_t(1) << lg) < c->page_size) ++lg;
  *out = {c->k_codes, c->k_scales, c->v_codes, c->v_scales, c->k_gscale, c->v_gscale, c->num_pages, lg,
          (int32_t)c->kv_heads, (int32_t)c->head_dim};
  return NVFP4_OK;
}

// The cache's buffers as ranges r[0..3] and its global scales as r[4..5].
void cache_ranges(const nvfp4_kv_cache& c, Range* r) {
  const int64_t n = c.num_pages * c.page_size * c.kv_heads * c.head_dim;
  r[0] = {c.k_codes, n / 2, "k_codes"};
  r[1] = {c.k_scales, n / 16, "k_scales"};
  r[2] = {c.v_codes, n / 2, "v_codes"};
  r[3] = {c.v_scales, n / 16, "v_scales"};
  r[4] = {c.k_gscale, 4, "k_gscale"};
  r[5] = {c.v_gscale, 4, "v_gscale"};
}

// A strided bf16 operand of `tokens` rows of `width` values; with no rows it
// may be null (an empty tensor's address).
nvfp4_status check_rows(const void* p, const char* name, int64_t stride, int64_t width, int64_t tokens) {
  if (p == nullptr && tokens > 0) return fail(NVFP4_ERR_INVALID_ARG, "%s is a null pointer", name);
  if (!aligned(p, 16)) return fail(NVFP4_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  if (stride < width) return fail(NVFP4_ERR_SHAPE, "%s has token stride %lld below its row of %lld", name,
                                  (long long)stride, (long long)width);
  if (stride % 8 != 0) return fail(NVFP4_ERR_ALIGNMENT, "%s has token stride %lld, not a multiple of 8", name,
                                   (long long)stride);
  if (tokens > 0 && stride > kMaxElems / tokens)
    return fail(NVFP4_ERR_UNSUPPORTED, "%s exceeds 2^40 elements", name);
  return NVFP4_OK;
}

// One grid dimension holds every workgroup of a cache operator when the
// rows it walks stay below this.
constexpr int64_t kMaxKvRows = int64_t(1) << 31;

nvfp4_status check_norm_rope(const nvfp4k::NormRope& a, int64_t q_heads, int64_t k_heads, int64_t head_dim,
                             int64_t rot_dim) {
  if (nvfp4_status s = check_dims(q_heads, "q_heads", k_heads, "k_heads", a.tokens, "tokens")) return s;
  if (nvfp4_status s = check_dims(rot_dim, "rot_dim", a.max_pos, "max_pos", head_dim, "head_dim")) return s;
  if (!nvfp4k::kv_head_dim_supported(head_dim))
    return fail(NVFP4_ERR_UNSUPPORTED, "head_dim=%lld; supported head sizes are 64, 128 and 256", (long long)head_dim);
  if (q_heads < 1 || k_heads < 1 || q_heads + k_heads > 32768)
    return fail(NVFP4_ERR_UNSUPPORTED, "q_heads=%lld, k_heads=%lld; at least 1 each and at most 32768 in all are supported",
                (long long)q_heads, (long long)k_heads);
  if (rot_dim > head_dim || rot_dim % 8 != 0)
    return fail(NVFP4_ERR_SHAPE, "rot_dim=%lld is not a multiple of 8 up to head_dim=%lld", (long long)rot_dim,
                (long long)head_dim);
  if (!(a.eps >= 0.0f)) return fail(NVFP4_ERR_INVALID_ARG, "eps is negative or NaN");
  if (a.tokens * (q_heads + 2 * k_heads) >= kMaxKvRows)
    return fail(NVFP4_ERR_UNSUPPORTED, "tokens * heads exceeds 2^31 rows (tokens=%lld)", (long long)a.tokens);
  if (a.q_weight) REQUIRE_ALIGN(a.q_weight, 16);
  if (a.k_weight) REQUIRE_ALIGN(a.k_weight, 16);
  if (rot_dim > 0) {
    if (a.cos_sin == nullptr) return fail(NVFP4_ERR_INVALID_ARG, "cos_sin is a null pointer");
    if (a.positions == nullptr) return fail(NVFP4_ERR_INVALID_ARG, "positions is a null pointer");
    REQUIRE_ALIGN(a.cos_sin, 16);
    REQUIRE_ALIGN(a.positions, 4);
  }
  return NVFP4_OK;
}

// Output rows may be the operand they come from (same address and stride);
// any other sharing with an operand is refused.
nvfp4_status check_rows_disjoint(const void* o, const char* on, int64_t o_stride, int64_t o_width, const void* i,
                                 const char* in, int64_t i_stride, int64_t i_width, int64_t tokens, bool in_place) {
  if (in_place && o == i && o_stride == i_stride) return NVFP4_OK;
  if (strided_overlap(o, o_stride * 2, o_width * 2, i, i_stride * 2, i_width * 2, tokens))
    return fail(NVFP4_ERR_INVALID_ARG, "output %s overlaps input %s", on, in);
  return NVFP4_OK;
}

// The sizes that fix an attention call's work and workspace.
nvfp4_status check_attention(const nvfp4k::KvCache& c, int64_t q_heads, int64_t batch, int64_t total_q,
                             int64_t max_q_len, int64_t max_kv_len, int64_t prefix_len, nvfp4k::KvAttention* a) {
  if (nvfp4_status s = check_dims(q_heads, "q_heads", batch, "batch", total_q, "total_q")) return s;
  if (nvfp4_status s = check_dims(max_q_len, "max_q_len", max_kv_len, "max_kv_len", prefix_len, "prefix_len"))
    return s;
  if (q_heads < 1 || q_heads > 65535 || q_heads % c.heads != 0)
    return fail(NVFP4_ERR_SHAPE, "q_heads=%lld is not a multiple of kv_heads=%d up to 65535", (long long)q_heads, c.heads);
  if (total_q > 0 && (batch < 1 || max_q_len < 1))
    return fail(NVFP4_ERR_INVALID_ARG, "batch=%lld and max_q_len=%lld must be positive with total_q=%lld",
                (long long)batch, (long long)max_q_len, (long long)total_q);
  if (total_q > batch * max_q_len)
    return fail(NVFP4_ERR_INVALID_ARG, "total_q=%lld: q_starts cannot lay them out in batch=%lld sequences of at most max_q_len=%lld",
                (long long)total_q, (long long)batch, (long long)max_q_len);
  if (total_q * q_heads >= kMaxKvRows)
    return fail(NVFP4_ERR_UNSUPPORTED, "total_q * q_heads exceeds 2^31 rows (total_q=%lld)", (long long)total_q);
  // key positions and the look-ahead past them stay in int
  if (max_kv_len + prefix_len > (int64_t(1) << 30))
    return fail(NVFP4_ERR_UNSUPPORTED, "prefix_len + max_kv_len exceeds 2^30 tokens");
  a->batch = (int32_t)batch;
  a->total_q = total_q;
  a->q_heads = (int32_t)q_heads;
  // no sequence has more queries than there are rows: with that the row tiles
  // of a sequence stay in int, as total_q * q_heads does
  a->max_q_len = (int32_t)(max_q_len < total_q ? max_q_len : total_q);
  a->max_kv_len = (int32_t)max_kv_len;
  a->prefix_len = (int32_t)prefix_len;
  if (total_q > 0 && !nvfp4k::kv_attention_supported(c, *a))
    return fail(NVFP4_ERR_UNSUPPORTED, "the call is too large (batch=%lld, total_q=%lld, max_kv_len=%lld)",
                (long long)batch, (long long)total_q, (long long)max_kv_len);
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int nvfp4_abi_version(void) { return 1; }

size_t nvfp4_quantize_workspace_bytes(void) { return sizeof(uint32_t) * nvfp4k::kAmaxPartials; }

size_t nvfp4_quantize_lora_workspace_bytes(int64_t rows, int64_t cols, int64_t r) {
  if (rows < 0 || cols < 0 || r < 0 || rows > kMaxDim || cols > kMaxDim || r > nvfp4k::kLoraMaxRank) return 0;
  return (size_t)nvfp4k::lora_workspace_bytes(rows, cols, r);
}

const char* nvfp4_status_string(nvfp4_status s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_ERR_SHAPE: return "shape violates the format";
    case NVFP4_ERR_ALIGNMENT: return "misaligned pointer";
    case NVFP4_ERR_UNSUPPORTED: return "unsupported request";
    case NVFP4_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

const char* nvfp4_last_error(void) { return g_last_error; }

nvfp4_status nvfp4_quantize_ex(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                               float* global_scale, int use_given_global_scale, int scale_rule, void* workspace,
                               void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  REQUIRE_PTR(global_scale);
  if (!use_given_global_scale) REQUIRE_PTR(workspace);
  if (scale_rule < NVFP4_SCALE_ABSMAX || scale_rule > NVFP4_SCALE_MSE)
    return fail(NVFP4_ERR_INVALID_ARG, "unknown scale rule %d", scale_rule);
  if (nvfp4_status s = check_dims(rows, "rows", cols, "cols", 0, "-")) return s;
  if (cols % 16 != 0) return fail(NVFP4_ERR_SHAPE, "cols=%lld is not a multiple of 16", (long long)cols);
  if (rows > 0 && cols > INT64_MAX / 2 / rows) return fail(NVFP4_ERR_UNSUPPORTED, "rows*cols overflows");
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(codes, 16);
  REQUIRE_ALIGN(scales, 16);
  REQUIRE_ALIGN(global_scale, 4);
  if (!use_given_global_scale) REQUIRE_ALIGN(workspace, 4);
  const int64_t n = rows * cols;
  const Range outs[3] = {{codes, n / 2, "codes"}, {scales, n / 16, "scales"}, {global_scale, 4, "global_scale"}};
  const Range ins[2] = {{x_bf16, n * 2, "x"},
                        {workspace, use_given_global_scale ? 0 : (int64_t)nvfp4_quantize_workspace_bytes(),
                         "workspace"}};
  if (n == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 3, ins, 2)) return s;
  return hip_status(nvfp4k::launch_nvfp4_quantize(x_bf16, rows, cols, codes, scales, global_scale,
                                                  use_given_global_scale, scale_rule, (uint32_t*)workspace,
                                                  (hipStream_t)stream),
                    "nvfp4_quantize launch");
}

nvfp4_status nvfp4_quantize(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                            float* global_scale, int use_given_global_scale, void* workspace, void* stream) {
  return nvfp4_quantize_ex(x_bf16, rows, cols, codes, scales, global_scale, use_given_global_scale,
                           NVFP4_SCALE_ABSMAX, workspace, stream);
}

nvfp4_status nvfp4_quantize_noalloc(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                                    float* global_scale, int use_given_global_scale, void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  REQUIRE_PTR(global_scale);
  if (nvfp4_status s = check_dims(rows, "rows", cols, "cols", 0, "-")) return s;
  if (cols % 16 != 0) return fail(NVFP4_ERR_SHAPE, "cols=%lld is not a multiple of 16", (long long)cols);
  if (rows > 0 && cols > kMaxElems / rows) return fail(NVFP4_ERR_UNSUPPORTED, "rows*cols exceeds 2^40");
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(codes, 16);
  REQUIRE_ALIGN(scales, 16);
  REQUIRE_ALIGN(global_scale, 4);
  const int64_t n = rows * cols;
  const Range outs[3] = {{codes, n / 2, "codes"}, {scales, n / 16, "scales"}, {global_scale, 4, "global_scale"}};
  const Range ins[1] = {{x_bf16, n * 2, "x"}};
  if (n == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 3, ins, 1)) return s;
  // the first pass writes at most kAmaxPartials partial maxima, which is
  // exactly the scratch's size, for every input size accepted above
  uint32_t* partials = nullptr;
  if (!use_given_global_scale) {
    const hipError_t e = nvfp4k::quantize_scratch((hipStream_t)stream, &partials);
    if (e != hipSuccess) return hip_status(e, "nvfp4_quantize_noalloc scratch lookup");
  }
  return hip_status(nvfp4k::launch_nvfp4_quantize(x_bf16, rows, cols, codes, scales, global_scale,
                                                  use_given_global_scale, NVFP4_SCALE_ABSMAX, partials,
                                                  (hipStream_t)stream),
                    "nvfp4_quantize_noalloc launch");
}

nvfp4_status nvfp4_gemm_ex(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                           const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale, void* out_bf16,
                           int64_t M, int64_t N, int64_t K, int algo, void* stream) {
  return gemm_impl(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K, algo, nullptr,
                   nullptr, 0, nullptr, 0, stream);
}

size_t nvfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 16 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K >= kTiledKLimit) return 0;
  return (size_t)nvfp4k::nvfp4_gemm_tiled_workspace_bytes(M, N, K);
}

nvfp4_status nvfp4_gemm_ws(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                           const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale, void* out_bf16,
                           int64_t M, int64_t N, int64_t K, int algo, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return gemm_impl(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K, algo, nullptr,
                   nullptr, 0, workspace, workspace_bytes, stream);
}

size_t nvfp4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N < 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
  if (nvfp4k::nvfp4_linear_fused_supported(M, K)) return 0;
  // the quantizer's partial maxima, then (stream-ordered, after the
  // quantizer is done with them) the GEMM's split-K partial sums
  const size_t g = nvfp4_gemm_workspace_bytes(M, N, K), q = nvfp4_quantize_workspace_bytes();
  return g > q ? g : q;
}

nvfp4_status nvfp4_linear(const void* x_bf16, const uint8_t* w_codes, const uint8_t* w_scales,
                          const float* w_gscale, void* out_bf16, int64_t M, int64_t N, int64_t K, uint8_t* x_codes,
                          uint8_t* x_scales, float* x_gscale, void* workspace, size_t workspace_bytes, void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(w_codes);
  REQUIRE_PTR(w_scales);
  REQUIRE_PTR(w_gscale);
  REQUIRE_PTR(out_bf16);
  REQUIRE_PTR(x_codes);
  REQUIRE_PTR(x_scales);
  REQUIRE_PTR(x_gscale);
  if (nvfp4_status s = check_dims(M, "M", N, "N", K, "K")) return s;
  if (nvfp4_status s = check_products(M, N, K)) return s;
  if (K <= 0 || K % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "K=%lld is not a positive multiple of 16", (long long)K);
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(w_codes, 16);
  REQUIRE_ALIGN(w_scales, 16);
  REQUIRE_ALIGN(w_gscale, 4);
  REQUIRE_ALIGN(out_bf16, 16);
  REQUIRE_ALIGN(x_codes, 16);
  REQUIRE_ALIGN(x_scales, 16);
  REQUIRE_ALIGN(x_gscale, 4);
  const size_t need = nvfp4_linear_workspace_bytes(M, N, K);
  if (need > 0) {
    REQUIRE_PTR(workspace);
    REQUIRE_ALIGN(workspace, 256);
    if (workspace_bytes < need)
      return fail(NVFP4_ERR_INVALID_ARG, "workspace_bytes=%zu is below nvfp4_linear_workspace_bytes=%zu",
                  workspace_bytes, need);
  }
  const Range outs[5] = {{out_bf16, M * N * 2, "out"},
                         {x_codes, M * K / 2, "x_codes"},
                         {x_scales, M * K / 16, "x_scales"},
                         {x_gscale, 4, "x_gscale"},
                         {workspace, need > 0 ? (int64_t)need : 0, "workspace"}};
  const Range ins[4] = {{x_bf16, M * K * 2, "x"},
                        {w_codes, N * K / 2, "w_codes"},
                        {w_scales, N * K / 16, "w_scales"},
                        {w_gscale, 4, "w_gscale"}};
  if (M == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 5, ins, 4)) return s;
  hipStream_t st = (hipStream_t)stream;
  if (N > 0 && nvfp4k::nvfp4_linear_fused_supported(M, K))
    return hip_status(nvfp4k::launch_nvfp4_linear_fused(x_bf16, w_codes, w_scales, w_gscale, out_bf16, M, N, K,
                                                        x_codes, x_scales, x_gscale, st),
                      "nvfp4_linear fused launch");
  nvfp4_status s = hip_status(nvfp4k::launch_nvfp4_quantize(x_bf16, M, K, x_codes, x_scales, x_gscale, 0,
                                                             NVFP4_SCALE_ABSMAX, (uint32_t*)workspace, st),
                              "nvfp4_linear quantize launch");
  if (s != NVFP4_OK || N == 0) return s;
  return gemm_impl(x_codes, x_scales, x_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K, NVFP4_ALGO_AUTO,
                   nullptr, nullptr, 0, workspace, workspace_bytes, stream);
}

size_t nvfp4_gemm_amax_slots(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K < 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim) return 0;
  if (check_products(M, N, K) != NVFP4_OK) return 0;
  return (size_t)amax_slots(M, N, K);
}

nvfp4_status nvfp4_gemm_amax(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                             const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale, void* out_bf16,
                             int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                             uint32_t* amax_slots, void* stream) {
  REQUIRE_PTR(amax_slots);
  REQUIRE_ALIGN(amax_slots, 4);
  if (N % 16 != 0)
    return fail(NVFP4_ERR_SHAPE, "N=%lld is not a multiple of 16 (the output is quantized along N)", (long long)N);
  return gemm_impl(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K, NVFP4_ALGO_AUTO,
                   nullptr, nullptr, 0, workspace, workspace_bytes, stream, amax_slots);
}

nvfp4_status nvfp4_quantize_amax(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                                 float* global_scale, const uint32_t* amax_slots, int64_t nslots, void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  REQUIRE_PTR(global_scale);
  REQUIRE_PTR(amax_slots);
  if (nvfp4_status s = check_dims(rows, "rows", cols, "cols", nslots, "nslots")) return s;
  if (nslots < 1 || nslots > (int64_t(1) << 28))
    return fail(NVFP4_ERR_INVALID_ARG, "nslots=%lld is outside [1, 2^28]", (long long)nslots);
  if (cols % 16 != 0) return fail(NVFP4_ERR_SHAPE, "cols=%lld is not a multiple of 16", (long long)cols);
  if (rows > 0 && cols > kMaxElems / rows) return fail(NVFP4_ERR_UNSUPPORTED, "rows*cols exceeds 2^40");
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(codes, 16);
  REQUIRE_ALIGN(scales, 16);
  REQUIRE_ALIGN(global_scale, 4);
  REQUIRE_ALIGN(amax_slots, 4);
  const int64_t n = rows * cols;
  const Range outs[3] = {{codes, n / 2, "codes"}, {scales, n / 16, "scales"}, {global_scale, 4, "global_scale"}};
  const Range ins[2] = {{x_bf16, n * 2, "x"}, {amax_slots, 4 * nslots, "amax_slots"}};
  if (n == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 3, ins, 2)) return s;
  return hip_status(nvfp4k::launch_nvfp4_quantize_pass2(x_bf16, rows, cols, codes, scales, global_scale, 0,
                                                        nvfp4k::kRuleAbsmax, (int)nslots,
                                                        const_cast<uint32_t*>(amax_slots), (hipStream_t)stream),
                    "nvfp4_quantize_amax launch");
}

nvfp4_status nvfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                        const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale, void* out_bf16,
                        int64_t M, int64_t N, int64_t K, void* stream) {
  return nvfp4_gemm_ex(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K,
                       NVFP4_ALGO_AUTO, stream);
}

nvfp4_status nvfp4_gemm_w4a16_ex(const void* x_bf16, const uint8_t* w_codes, const uint8_t* w_scales,
                                 const float* w_gscale, void* out_bf16, int64_t M, int64_t N, int64_t K, int algo,
                                 void* stream) {
  if (nvfp4_status s = check_dims(M, "M", N, "N", K, "K")) return s;
  if (nvfp4_status s = check_products(M, N, K)) return s;
  if (K > 0) {
    REQUIRE_PTR(x_bf16);
    REQUIRE_PTR(w_codes);
    REQUIRE_PTR(w_scales);
  }
  REQUIRE_PTR(w_gscale);
  REQUIRE_PTR(out_bf16);
  if (K % 16 != 0) return fail(NVFP4_ERR_SHAPE, "K=%lld is not a multiple of 16", (long long)K);
  if (algo < NVFP4_ALGO_AUTO || algo > NVFP4_ALGO_SIMPLE) return fail(NVFP4_ERR_INVALID_ARG, "unknown algo %d", algo);
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(w_codes, 16);
  REQUIRE_ALIGN(w_scales, 16);
  REQUIRE_ALIGN(out_bf16, 16);
  REQUIRE_ALIGN(w_gscale, 4);
  const Range outs[1] = {{out_bf16, M * N * 2, "out"}};
  const Range ins[4] = {{x_bf16, M * K * 2, "x"}, {w_codes, N * K / 2, "w_codes"},
                        {w_scales, N * K / 16, "w_scales"}, {w_gscale, 4, "w_gscale"}};
  if (M == 0 || N == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 1, ins, 4)) return s;
  const bool decode_ok = nvfp4k::nvfp4_w4a16_decode_supported(M, K);
  // the tiled kernel stages 128 values per step and addresses a tile's rows
  // of x (128 x 2K bytes) with 32-bit buffer offsets
  const bool tiled_ok = K > 0 && K % 128 == 0 && K < kInt4TiledKLimit;
  if (algo == NVFP4_ALGO_AUTO)
    algo = decode_ok ? NVFP4_ALGO_DECODE : (tiled_ok ? NVFP4_ALGO_TILED : NVFP4_ALGO_SIMPLE);
  hipStream_t st = (hipStream_t)stream;
  if (algo == NVFP4_ALGO_TILED) {
    if (!tiled_ok)
      return fail(NVFP4_ERR_UNSUPPORTED, "weight-only tiled kernel needs K %% 128 == 0 and 0 < K < 2^22 (K=%lld)",
                  (long long)K);
    return hip_status(nvfp4k::launch_nvfp4_w4a16_tiled(x_bf16, w_codes, w_scales, w_gscale, out_bf16, M, N, K, st),
                      "nvfp4_gemm_w4a16 tiled launch");
  }
  if (algo == NVFP4_ALGO_DECODE) {
    if (!decode_ok)
      return fail(NVFP4_ERR_UNSUPPORTED, "weight-only decode kernel needs M <= 16, K %% 128 == 0 and K <= 32768 "
                  "(M=%lld, K=%lld)", (long long)M, (long long)K);
    return hip_status(nvfp4k::launch_nvfp4_w4a16_decode(x_bf16, w_codes, w_scales, w_gscale, out_bf16, M, N, K, st),
                      "nvfp4_gemm_w4a16 decode launch");
  }
  return hip_status(nvfp4k::launch_nvfp4_w4a16_simple(x_bf16, w_codes, w_scales, w_gscale, out_bf16, M, N, K, st),
                    "nvfp4_gemm_w4a16 simple launch");
}

nvfp4_status nvfp4_gemm_w4a16(const void* x_bf16, const uint8_t* w_codes, const uint8_t* w_scales,
                              const float* w_gscale, void* out_bf16, int64_t M, int64_t N, int64_t K, void* stream) {
  return nvfp4_gemm_w4a16_ex(x_bf16, w_codes, w_scales, w_gscale, out_bf16, M, N, K, NVFP4_ALGO_AUTO, stream);
}

nvfp4_status int4g_quantize(const void* w_bf16, int64_t N, int64_t K, int64_t group, uint8_t* q, void* scales_fp16,
                            void* stream) {
  REQUIRE_PTR(w_bf16);
  REQUIRE_PTR(q);
  REQUIRE_PTR(scales_fp16);
  if (nvfp4_status s = check_dims(N, "N", K, "K", group, "group")) return s;
  if (group != 128) return fail(NVFP4_ERR_UNSUPPORTED, "group=%lld; only 128 is supported", (long long)group);
  if (K % 128 != 0) return fail(NVFP4_ERR_SHAPE, "K=%lld is not a multiple of the group (128)", (long long)K);
  REQUIRE_ALIGN(w_bf16, 16);
  REQUIRE_ALIGN(q, 16);
  REQUIRE_ALIGN(scales_fp16, 16);
  const Range outs[2] = {{q, N * K / 2, "q"}, {scales_fp16, N * (K / 128) * 2, "scales"}};
  const Range ins[1] = {{w_bf16, N * K * 2, "w"}};
  if (N == 0 || K == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 2, ins, 1)) return s;
  return hip_status(nvfp4k::launch_int4g_quantize(w_bf16, N, K, q, scales_fp16, (hipStream_t)stream),
                    "int4g_quantize launch");
}

nvfp4_status int4g_gemv_ex(const void* x_bf16, const uint8_t* q, const void* scales_fp16, void* out_bf16, int64_t M,
                           int64_t N, int64_t K, int64_t group, int algo, void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(q);
  REQUIRE_PTR(scales_fp16);
  REQUIRE_PTR(out_bf16);
  if (nvfp4_status s = check_dims(M, "M", N, "N", K, "K")) return s;
  if (nvfp4_status s = check_products(M, N, K)) return s;
  if (group != 128) return fail(NVFP4_ERR_UNSUPPORTED, "group=%lld; only 128 is supported", (long long)group);
  if (K % 128 != 0) return fail(NVFP4_ERR_SHAPE, "K=%lld is not a multiple of the group (128)", (long long)K);
  if (algo < NVFP4_ALGO_AUTO || algo > NVFP4_ALGO_SIMPLE) return fail(NVFP4_ERR_INVALID_ARG, "unknown algo %d", algo);
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(q, 16);
  REQUIRE_ALIGN(scales_fp16, 16);
  REQUIRE_ALIGN(out_bf16, 16);
  const Range outs[1] = {{out_bf16, M * N * 2, "out"}};
  const Range ins[3] = {{x_bf16, M * K * 2, "x"}, {q, N * K / 2, "q"}, {scales_fp16, N * (K / 128) * 2, "scales"}};
  if (M == 0 || N == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 1, ins, 3)) return s;
  if (algo == NVFP4_ALGO_AUTO)
    algo = (K == 0) ? NVFP4_ALGO_SIMPLE
                    : (M <= 16 ? (K <= kDecodeMaxK ? NVFP4_ALGO_DECODE : NVFP4_ALGO_SIMPLE)
                               : (K < kInt4TiledKLimit ? NVFP4_ALGO_TILED : NVFP4_ALGO_SIMPLE));
  hipStream_t st = (hipStream_t)stream;
  switch (algo) {
    case NVFP4_ALGO_TILED:
      if (K == 0 || K >= kInt4TiledKLimit)
        return fail(NVFP4_ERR_UNSUPPORTED, "tiled kernel needs 0 < K < 2^22 (K=%lld)", (long long)K);
      return hip_status(nvfp4k::launch_int4g_gemm_tiled(x_bf16, q, scales_fp16, out_bf16, M, N, K, st),
                        "int4g_gemv tiled launch");
    case NVFP4_ALGO_DECODE:
      if (M > 16 || K == 0 || K > kDecodeMaxK)
        return fail(NVFP4_ERR_UNSUPPORTED, "decode kernel needs M <= 16 and 0 < K <= 2^24 (M=%lld, K=%lld)",
                    (long long)M, (long long)K);
      return hip_status(nvfp4k::launch_int4g_gemm_decode(x_bf16, q, scales_fp16, out_bf16, M, N, K, st),
                        "int4g_gemv decode launch");
    default:
      return hip_status(nvfp4k::launch_int4g_gemm_simple(x_bf16, q, scales_fp16, out_bf16, M, N, K, st),
                        "int4g_gemv simple launch");
  }
}

nvfp4_status int4g_gemv(const void* x_bf16, const uint8_t* q, const void* scales_fp16, void* out_bf16, int64_t M,
                        int64_t N, int64_t K, int64_t group, void* stream) {
  return int4g_gemv_ex(x_bf16, q, scales_fp16, out_bf16, M, N, K, group, NVFP4_ALGO_AUTO, stream);
}

nvfp4_status int4g_asym_quantize(const void* w_bf16, int64_t N, int64_t K, int64_t group, uint8_t* q,
                                 void* scales_fp16, uint8_t* zeros, void* stream) {
  REQUIRE_PTR(w_bf16);
  REQUIRE_PTR(q);
  REQUIRE_PTR(scales_fp16);
  REQUIRE_PTR(zeros);
  if (nvfp4_status s = check_dims(N, "N", K, "K", group, "group")) return s;
  if (group != 128) return fail(NVFP4_ERR_UNSUPPORTED, "group=%lld; only 128 is supported", (long long)group);
  if (K % 128 != 0) return fail(NVFP4_ERR_SHAPE, "K=%lld is not a multiple of the group (128)", (long long)K);
  REQUIRE_ALIGN(w_bf16, 16);
  REQUIRE_ALIGN(q, 16);
  REQUIRE_ALIGN(scales_fp16, 16);
  const Range outs[3] = {{q, N * K / 2, "q"}, {scales_fp16, N * (K / 128) * 2, "scales"},
                         {zeros, N * (K / 128), "zeros"}};
  const Range ins[1] = {{w_bf16, N * K * 2, "w"}};
  if (N == 0 || K == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 3, ins, 1)) return s;
  return hip_status(nvfp4k::launch_int4g_asym_quantize(w_bf16, N, K, q, scales_fp16, zeros, (hipStream_t)stream),
                    "int4g_asym_quantize launch");
}

nvfp4_status int4g_asym_gemv_ex(const void* x_bf16, const uint8_t* q, const void* scales_fp16, const uint8_t* zeros,
                                void* out_bf16, int64_t M, int64_t N, int64_t K, int64_t group, int algo,
                                void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(q);
  REQUIRE_PTR(scales_fp16);
  REQUIRE_PTR(zeros);
  REQUIRE_PTR(out_bf16);
  if (nvfp4_status s = check_dims(M, "M", N, "N", K, "K")) return s;
  if (nvfp4_status s = check_products(M, N, K)) return s;
  if (group != 128) return fail(NVFP4_ERR_UNSUPPORTED, "group=%lld; only 128 is supported", (long long)group);
  if (K % 128 != 0) return fail(NVFP4_ERR_SHAPE, "K=%lld is not a multiple of the group (128)", (long long)K);
  if (algo < NVFP4_ALGO_AUTO || algo > NVFP4_ALGO_SIMPLE) return fail(NVFP4_ERR_INVALID_ARG, "unknown algo %d", algo);
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(q, 16);
  REQUIRE_ALIGN(scales_fp16, 16);
  REQUIRE_ALIGN(out_bf16, 16);
  const Range outs[1] = {{out_bf16, M * N * 2, "out"}};
  const Range ins[4] = {{x_bf16, M * K * 2, "x"}, {q, N * K / 2, "q"}, {scales_fp16, N * (K / 128) * 2, "scales"},
                        {zeros, N * (K / 128), "zeros"}};
  if (M == 0 || N == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 1, ins, 4)) return s;
  const bool decode_ok = nvfp4k::int4g_asym_decode_supported(M, K);
  if (algo == NVFP4_ALGO_AUTO)
    algo = decode_ok ? NVFP4_ALGO_DECODE : (K < kInt4TiledKLimit ? NVFP4_ALGO_TILED : NVFP4_ALGO_SIMPLE);
  hipStream_t st = (hipStream_t)stream;
  if (algo == NVFP4_ALGO_TILED) {
    if (K >= kInt4TiledKLimit)
      return fail(NVFP4_ERR_UNSUPPORTED, "tiled kernel needs 0 < K < 2^22 (K=%lld)", (long long)K);
    return hip_status(nvfp4k::launch_int4g_asym_tiled(x_bf16, q, scales_fp16, zeros, out_bf16, M, N, K, st),
                      "int4g_asym_gemv tiled launch");
  }
  if (algo == NVFP4_ALGO_DECODE) {
    if (!decode_ok)
      return fail(NVFP4_ERR_UNSUPPORTED, "asymmetric decode kernel needs M <= 2 and 0 < K <= 32768 (M=%lld, K=%lld)",
                  (long long)M, (long long)K);
    return hip_status(nvfp4k::launch_int4g_asym_decode(x_bf16, q, scales_fp16, zeros, out_bf16, M, N, K, st),
                      "int4g_asym_gemv decode launch");
  }
  return hip_status(nvfp4k::launch_int4g_asym_simple(x_bf16, q, scales_fp16, zeros, out_bf16, M, N, K, st),
                    "int4g_asym_gemv simple launch");
}

nvfp4_status int4g_asym_gemv(const void* x_bf16, const uint8_t* q, const void* scales_fp16, const uint8_t* zeros,
                             void* out_bf16, int64_t M, int64_t N, int64_t K, int64_t group, void* stream) {
  return int4g_asym_gemv_ex(x_bf16, q, scales_fp16, zeros, out_bf16, M, N, K, group, NVFP4_ALGO_AUTO, stream);
}

nvfp4_status nvfp4_quantize_lora(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                                 float* global_scale, int use_given_global_scale, const void* lora_down_bf16,
                                 int64_t r, float* lora_t, void* workspace, void* stream) {
  REQUIRE_PTR(x_bf16);
  REQUIRE_PTR(codes);
  REQUIRE_PTR(scales);
  REQUIRE_PTR(global_scale);
  REQUIRE_PTR(lora_down_bf16);
  REQUIRE_PTR(lora_t);
  REQUIRE_PTR(workspace);
  if (nvfp4_status s = check_dims(rows, "rows", cols, "cols", r, "r")) return s;
  if (nvfp4_status s = check_rank(r)) return s;
  if (cols % 16 != 0) return fail(NVFP4_ERR_SHAPE, "cols=%lld is not a multiple of 16", (long long)cols);
  if (rows > 0 && cols > INT64_MAX / 2 / rows) return fail(NVFP4_ERR_UNSUPPORTED, "rows*cols overflows");
  if (r * cols * 2 > (int64_t)INT32_MAX || 16 * cols * 2 > (int64_t)INT32_MAX)
    return fail(NVFP4_ERR_UNSUPPORTED, "r*cols or 16*cols exceeds 2^30 values (r=%lld, cols=%lld)", (long long)r,
                (long long)cols);
  REQUIRE_ALIGN(x_bf16, 16);
  REQUIRE_ALIGN(codes, 16);
  REQUIRE_ALIGN(scales, 16);
  REQUIRE_ALIGN(global_scale, 4);
  REQUIRE_ALIGN(lora_down_bf16, 16);
  REQUIRE_ALIGN(lora_t, 16);
  REQUIRE_ALIGN(workspace, 4);
  const int64_t n = rows * cols;
  const Range outs[4] = {{codes, n / 2, "codes"}, {scales, n / 16, "scales"}, {global_scale, 4, "global_scale"},
                         {lora_t, rows * r * 4, "lora_t"}};
  const Range ins[3] = {{x_bf16, n * 2, "x"}, {lora_down_bf16, r * cols * 2, "lora_down"},
                        {workspace, nvfp4k::lora_workspace_bytes(rows, cols, r), "workspace"}};
  if (rows == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 4, ins, 3)) return s;
  return hip_status(nvfp4k::launch_nvfp4_quantize_lora(x_bf16, rows, cols, codes, scales, global_scale,
                                                       use_given_global_scale, lora_down_bf16, r, lora_t,
                                                       (uint32_t*)workspace, (hipStream_t)stream),
                    "nvfp4_quantize_lora launch");
}

nvfp4_status nvfp4_gemm_lora_ex(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                                const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale,
                                const float* lora_t, const void* lora_up_bf16, int64_t r, void* out_bf16, int64_t M,
                                int64_t N, int64_t K, int algo, void* stream) {
  REQUIRE_PTR(lora_t);
  REQUIRE_PTR(lora_up_bf16);
  if (nvfp4_status s = check_dims(M, "M", N, "N", r, "r")) return s;
  if (nvfp4_status s = check_rank(r)) return s;
  if (M * r * 4 > (int64_t)INT32_MAX || N * r * 2 > (int64_t)INT32_MAX)
    return fail(NVFP4_ERR_UNSUPPORTED, "lora_t or lora_up exceeds 2 GiB (M=%lld, N=%lld, r=%lld)", (long long)M,
                (long long)N, (long long)r);
  REQUIRE_ALIGN(lora_t, 16);
  REQUIRE_ALIGN(lora_up_bf16, 16);
  return gemm_impl(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, out_bf16, M, N, K, algo, lora_t,
                   lora_up_bf16, r, nullptr, 0, stream);
}

nvfp4_status nvfp4_gemm_lora(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                             const uint8_t* w_codes, const uint8_t* w_scales, const float* w_gscale,
                             const float* lora_t, const void* lora_up_bf16, int64_t r, void* out_bf16, int64_t M,
                             int64_t N, int64_t K, void* stream) {
  return nvfp4_gemm_lora_ex(a_codes, a_scales, a_gscale, w_codes, w_scales, w_gscale, lora_t, lora_up_bf16, r,
                            out_bf16, M, N, K, NVFP4_ALGO_AUTO, stream);
}

nvfp4_status nvfp4_kv_write(const nvfp4_kv_cache* cache, const void* k_bf16, int64_t k_stride, const void* v_bf16,
                            int64_t v_stride, const int64_t* slots, int64_t tokens, void* stream) {
  nvfp4k::KvCache c;
  if (nvfp4_status s = check_cache(cache, &c)) return s;
  if (nvfp4_status s = check_dims(tokens, "tokens", 0, "-", 0, "-")) return s;
  const int64_t width = cache->kv_heads * cache->head_dim;
  if (nvfp4_status s = check_rows(k_bf16, "k", k_stride, width, tokens)) return s;
  if (nvfp4_status s = check_rows(v_bf16, "v", v_stride, width, tokens)) return s;
  if (tokens > 0) REQUIRE_PTR(slots);
  REQUIRE_ALIGN(slots, 8);
  if (tokens * 2 * cache->kv_heads >= kMaxKvRows)
    return fail(NVFP4_ERR_UNSUPPORTED, "tokens * heads exceeds 2^31 rows (tokens=%lld)", (long long)tokens);
  Range r[6];
  cache_ranges(*cache, r);
  const Range ins[5] = {{k_bf16, strided_bytes(tokens, k_stride * 2, width * 2), "k"},
                        {v_bf16, strided_bytes(tokens, v_stride * 2, width * 2), "v"},
                        {slots, tokens * 8, "slots"}, r[4], r[5]};
  if (tokens == 0 || cache->num_pages == 0) return ok();
  if (nvfp4_status s = check_disjoint(r, 4, ins, 5)) return s;
  return hip_status(nvfp4k::launch_kv_write(c, k_bf16, k_stride, v_bf16, v_stride, slots, tokens, (hipStream_t)stream),
                    "nvfp4_kv_write launch");
}

nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_bf16,
                           void* v_bf16, void* stream) {
  nvfp4k::KvCache c;
  if (nvfp4_status s = check_cache(cache, &c)) return s;
  if (nvfp4_status s = check_dims(tokens, "tokens", 0, "-", 0, "-")) return s;
  const int64_t width = cache->kv_heads * cache->head_dim;
  if (nvfp4_status s = check_rows(k_bf16, "k", width, width, tokens)) return s;
  if (nvfp4_status s = check_rows(v_bf16, "v", width, width, tokens)) return s;
  if (tokens > 0) REQUIRE_PTR(slots);
  REQUIRE_ALIGN(slots, 8);
  if (tokens * 2 * cache->kv_heads >= kMaxKvRows)
    return fail(NVFP4_ERR_UNSUPPORTED, "tokens * heads exceeds 2^31 rows (tokens=%lld)", (long long)tokens);
  Range ins[7];
  cache_ranges(*cache, ins);
  ins[6] = {slots, tokens * 8, "slots"};
  const Range outs[2] = {{k_bf16, tokens * width * 2, "k"}, {v_bf16, tokens * width * 2, "v"}};
  if (tokens == 0) return ok();
  if (nvfp4_status s = check_disjoint(outs, 2, ins, 7)) return s;
  return hip_status(nvfp4k::launch_kv_read(c, slots, tokens, k_bf16, v_bf16, (hipStream_t)stream),
                    "nvfp4_kv_read launch");
}

nvfp4_status nvfp4_qk_norm_rope(const void* q_bf16, int64_t q_stride, const void* q_weight_bf16, void* q_out_bf16,
                                int64_t q_out_stride, int64_t q_heads, const void* k_bf16, int64_t k_stride,
                                const void* k_weight_bf16, void* k_out_bf16, int64_t k_out_stride, int64_t k_heads,
                                int64_t head_dim, const float* cos_sin, int64_t max_pos, int64_t rot_dim,
                                int interleaved, const int32_t* positions, float eps, int64_t tokens, void* stream) {
  const nvfp4k::NormRope a{(const uint16_t*)q_bf16, (const uint16_t*)k_bf16, (const uint16_t*)q_weight_bf16,
                           (const uint16_t*)k_weight_bf16, (uint16_t*)q_out_bf16, (uint16_t*)k_out_bf16, q_stride,
                           k_stride, q_out_stride, k_out_stride, cos_sin, positions, tokens, max_pos,
                           (int32_t)q_heads, (int32_t)k_heads, (int32_t)rot_dim, interleaved != 0, eps, 0};
  if (nvfp4_status s = check_norm_rope(a, q_heads, k_heads, head_dim, rot_dim)) return s;
  const int64_t qw = q_heads * head_dim, kw = k_heads * head_dim;
  if (nvfp4_status s = check_rows(q_bf16, "q", q_stride, qw, tokens)) return s;
  if (nvfp4_status s = check_rows(k_bf16, "k", k_stride, kw, tokens)) return s;
  if (nvfp4_status s = check_rows(q_out_bf16, "q_out", q_out_stride, qw, tokens)) return s;
  if (nvfp4_status s = check_rows(k_out_bf16, "k_out", k_out_stride, kw, tokens)) return s;
  if (tokens == 0) return ok();
  if (nvfp4_status s = check_rows_disjoint(q_out_bf16, "q_out", q_out_stride, qw, q_bf16, "q", q_stride, qw, tokens, true)) return s;
  if (nvfp4_status s = check_rows_disjoint(q_out_bf16, "q_out", q_out_stride, qw, k_bf16, "k", k_stride, kw, tokens, false)) return s;
  if (nvfp4_status s = check_rows_disjoint(k_out_bf16, "k_out", k_out_stride, kw, k_bf16, "k", k_stride, kw, tokens, true)) return s;
  if (nvfp4_status s = check_rows_disjoint(k_out_bf16, "k_out", k_out_stride, kw, q_bf16, "q", q_stride, qw, tokens, false)) return s;
  if (nvfp4_status s = check_rows_disjoint(q_out_bf16, "q_out", q_out_stride, qw, k_out_bf16, "k_out", k_out_stride, kw, tokens, false)) return s;
  const Range outs[2] = {{q_out_bf16, strided_bytes(tokens, q_out_stride * 2, qw * 2), "q_out"},
                         {k_out_bf16, strided_bytes(tokens, k_out_stride * 2, kw * 2), "k_out"}};
  const Range ins[4] = {{q_weight_bf16, q_weight_bf16 ? head_dim * 2 : 0, "q_weight"},
                        {k_weight_bf16, k_weight_bf16 ? head_dim * 2 : 0, "k_weight"},
                        {cos_sin, max_pos * rot_dim * 4, "cos_sin"},
                        {positions, rot_dim ? tokens * 4 : 0, "positions"}};
  for (const Range& o : outs)
    if (nvfp4_status s = check_disjoint(&o, 1, ins, 4)) return s;
  return hip_status(nvfp4k::launch_norm_rope(a, (int)head_dim, nullptr, nullptr, nullptr, 0, (hipStream_t)stream),
                    "nvfp4_qk_norm_rope launch");
}

nvfp4_status nvfp4_qk_norm_rope_write(const nvfp4_kv_cache* cache, const void* q_bf16, int64_t q_stride,
                                      const void* q_weight_bf16, void* q_out_bf16, int64_t q_out_stride,
                                      int64_t q_heads, const void* k_bf16, int64_t k_stride,
                                      const void* k_weight_bf16, const void* v_bf16, int64_t v_stride,
                                      const float* cos_sin, int64_t max_pos, int64_t rot_dim, int interleaved,
                                      const int32_t* positions, float eps, const int64_t* slots, int64_t tokens,
                                      void* stream) {
  nvfp4k::KvCache c;
  if (nvfp4_status s = check_cache(cache, &c)) return s;
  const int64_t d = cache->head_dim, kh = cache->kv_heads;
  const nvfp4k::NormRope a{(const uint16_t*)q_bf16, (const uint16_t*)k_bf16, (const uint16_t*)q_weight_bf16,
                           (const uint16_t*)k_weight_bf16, (uint16_t*)q_out_bf16, nullptr, q_stride, k_stride,
                           q_out_stride, 0, cos_sin, positions, tokens, max_pos, (int32_t)q_heads, (int32_t)kh,
                           (int32_t)rot_dim, interleaved != 0, eps, 0};
  if (nvfp4_status s = check_norm_rope(a, q_heads, kh, d, rot_dim)) return s;
  const int64_t qw = q_heads * d, kw = kh * d;
  if (nvfp4_status s = check_rows(q_bf16, "q", q_stride, qw, tokens)) return s;
  if (nvfp4_status s = check_rows(k_bf16, "k", k_stride, kw, tokens)) return s;
  if (nvfp4_status s = check_rows(v_bf16, "v", v_stride, kw, tokens)) return s;
  if (nvfp4_status s = check_rows(q_out_bf16, "q_out", q_out_stride, qw, tokens)) return s;
  if (tokens > 0) REQUIRE_PTR(slots);
  REQUIRE_ALIGN(slots, 8);
  if (tokens == 0) return ok();
  if (nvfp4_status s = check_rows_disjoint(q_out_bf16, "q_out", q_out_stride, qw, q_bf16, "q", q_stride, qw, tokens, true)) return s;
  if (nvfp4_status s = check_rows_disjoint(q_out_bf16, "q_out", q_out_stride, qw, k_bf16, "k", k_stride, kw, tokens, false)) return s;
  if (nvfp4_status s = check_rows_disjoint(q_out_bf16, "q_out", q_out_stride, qw, v_bf16, "v", v_stride, kw, tokens, false)) return s;
  Range r[6];
  cache_ranges(*cache, r);
  const Range outs[5] = {r[0], r[1], r[2], r[3],
                         {q_out_bf16, strided_bytes(tokens, q_out_stride * 2, qw * 2), "q_out"}};
  const Range ins[7] = {{q_weight_bf16, q_weight_bf16 ? d * 2 : 0, "q_weight"},
                        {k_weight_bf16, k_weight_bf16 ? d * 2 : 0, "k_weight"},
                        {cos_sin, max_pos * rot_dim * 4, "cos_sin"},
                        {positions, rot_dim ? tokens * 4 : 0, "positions"},
                        {slots, tokens * 8, "slots"}, r[4], r[5]};
  if (nvfp4_status s = check_disjoint(outs, 5, ins, 7)) return s;
  const Range rows[3] = {{q_bf16, strided_bytes(tokens, q_stride * 2, qw * 2), "q"},
                         {k_bf16, strided_bytes(tokens, k_stride * 2, kw * 2), "k"},
                         {v_bf16, strided_bytes(tokens, v_stride * 2, kw * 2), "v"}};
  if (nvfp4_status s = check_disjoint(outs, 4, rows, 3)) return s;
  return hip_status(nvfp4k::launch_norm_rope(a, (int)d, &c, slots, v_bf16, v_stride, (hipStream_t)stream),
                    "nvfp4_qk_norm_rope_write launch");
}

size_t nvfp4_kv_attention_workspace_bytes(const nvfp4_kv_cache* cache, int64_t q_heads, int64_t batch,
                                          int64_t total_q, int64_t max_q_len, int64_t max_kv_len,
                                          int64_t prefix_len) {
  nvfp4k::KvCache c;
  nvfp4k::KvAttention a{};
  if (check_cache(cache, &c) != NVFP4_OK ||
      check_attention(c, q_heads, batch, total_q, max_q_len, max_kv_len, prefix_len, &a) != NVFP4_OK)
    return 0;
  return (size_t)nvfp4k::kv_attention_workspace_bytes(c, a);
}

nvfp4_status nvfp4_kv_attention(const nvfp4_kv_cache* cache, const void* q_bf16, int64_t q_stride, int64_t q_heads,
                                const int32_t* q_starts, int64_t batch, int64_t total_q, int64_t max_q_len,
                                const int32_t* page_table, int64_t table_width, const int32_t* kv_lens,
                                int64_t max_kv_len, const int32_t* prefix_pages, int64_t prefix_len, float scale,
                                void* out_bf16, void* workspace, size_t workspace_bytes, void* stream) {
  nvfp4k::KvCache c;
  nvfp4k::KvAttention a{};
  if (nvfp4_status s = check_cache(cache, &c)) return s;
  if (nvfp4_status s = check_attention(c, q_heads, batch, total_q, max_q_len, max_kv_len, prefix_len, &a)) return s;
  const int64_t width = q_heads * cache->head_dim;
  if (nvfp4_status s = check_rows(q_bf16, "q", q_stride, width, total_q)) return s;
  if (total_q > 0) {
    REQUIRE_PTR(kv_lens);
    REQUIRE_PTR(out_bf16);
    if (max_kv_len > 0) REQUIRE_PTR(page_table);
  }
  REQUIRE_ALIGN(kv_lens, 4);
  REQUIRE_ALIGN(out_bf16, 16);
  if (table_width < 0 || table_width > kMaxDim)
    return fail(NVFP4_ERR_INVALID_ARG, "table_width=%lld is out of range", (long long)table_width);
  if (max_kv_len > table_width * cache->page_size)
    return fail(NVFP4_ERR_SHAPE, "max_kv_len=%lld exceeds the page table's %lld pages of %lld tokens",
                (long long)max_kv_len, (long long)table_width, (long long)cache->page_size);
  REQUIRE_ALIGN(page_table, 4);
  if (prefix_len > 0) REQUIRE_PTR(prefix_pages);
  REQUIRE_ALIGN(prefix_pages, 4);
  if (q_starts == nullptr && (total_q != batch || max_q_len != 1))
    return fail(NVFP4_ERR_INVALID_ARG, "q_starts is null: total_q=%lld must equal batch=%lld and max_q_len=%lld be 1",
                (long long)total_q, (long long)batch, (long long)max_q_len);
  REQUIRE_ALIGN(q_starts, 4);
  if (!(scale > 0.0f) || scale > 1e30f) return fail(NVFP4_ERR_INVALID_ARG, "scale is not a positive finite number");
  const size_t need = (size_t)nvfp4k::kv_attention_workspace_bytes(c, a);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need)
      return fail(NVFP4_ERR_INVALID_ARG, "workspace holds %llu bytes, the call needs %llu",
                  (unsigned long long)(workspace ? workspace_bytes : 0), (unsigned long long)need);
    REQUIRE_ALIGN(workspace, 256);
  }
  if (total_q == 0) return ok();
  const int64_t prefix_count = (prefix_len + cache->page_size - 1) / cache->page_size;
  Range ins[11];
  cache_ranges(*cache, ins);
  ins[6] = {q_bf16, strided_bytes(total_q, q_stride * 2, width * 2), "q"};
  ins[7] = {page_table, batch * table_width * 4, "page_table"};
  ins[8] = {kv_lens, batch * 4, "kv_lens"};
  ins[9] = {prefix_pages, prefix_count * 4, "prefix_pages"};
  ins[10] = {q_starts, q_starts ? (batch + 1) * 4 : 0, "q_starts"};
  const Range outs[2] = {{out_bf16, total_q * width * 2, "out"}, {workspace, (int64_t)need, "workspace"}};
  if (nvfp4_status s = check_disjoint(outs, 2, ins, 11)) return s;
  a.q = (const uint16_t*)q_bf16;
  a.q_stride = q_stride;
  a.out = (uint16_t*)out_bf16;
  a.q_starts = q_starts;
  a.page_table = page_table;
  a.table_width = table_width;
  a.kv_lens = kv_lens;
  a.prefix_pages = prefix_pages;
  a.scale = scale;
  return hip_status(nvfp4k::launch_kv_attention(c, a, workspace, (hipStream_t)stream), "nvfp4_kv_attention launch");
}

}  // extern "C"
