// Host side of include/snip_kv.h: argument validation (before any HIP call)
// and kernel enqueueing for the 4-bit key/value cache and the attention over it.
#include <cmath>
#include <cstring>

#include "api_common.h"
#include "kv.h"

using namespace snip;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 20;
constexpr int64_t kMaxTiles = ((int64_t)1 << 24) - 1;   // of 256 threads in a grid's dimension
constexpr int64_t kMaxSeqs = (int64_t)1 << 20;
constexpr int64_t kMaxLen = (int64_t)1 << 30;          // of a table, in tokens
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxLd = (int64_t)1 << 40;            // times kMaxTokens and an element's bytes: within 63 bits

bool head_dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }

int check_cache(const char* who, const snipkv_cache* c, KvCache* v) {
  if (!c) return fail(SNIP_E_NULL, "%s: cache is NULL", who);
  if (c->format != SNIP_NVFP4 && c->format != SNIP_MXFP4)
    return fail(SNIP_E_FORMAT, "%s: cache format %d is not NVFP4 or MXFP4", who, c->format);
  if (c->page_size < 16 || c->page_size > SNIPKV_MAX_PAGE_SIZE || (c->page_size & (c->page_size - 1)))
    return fail(SNIP_E_SHAPE, "%s: page_size=%d must be a power of two in 16 .. %d", who, c->page_size,
                SNIPKV_MAX_PAGE_SIZE);
  if (c->kv_heads < 1 || c->kv_heads > kMaxHeads)
    return fail(SNIP_E_SHAPE, "%s: kv_heads=%d outside 1 .. %lld", who, c->kv_heads, (long long)kMaxHeads);
  if (!head_dim_ok(c->head_dim)) return fail(SNIP_E_SHAPE, "%s: head_dim=%d is not 64, 128 or 256", who, c->head_dim);
  if (c->pages < 1 || c->pages > INT32_MAX)
    return fail(SNIP_E_SHAPE, "%s: pages=%lld outside 1 .. 2^31 - 1", who, (long long)c->pages);
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales || (c->format == SNIP_NVFP4 && !c->texp))
    return fail(SNIP_E_NULL, "%s: the cache's buffers must be non-NULL", who);
  if (!aligned(c->k_codes, 16) || !aligned(c->k_scales, 16) || !aligned(c->v_codes, 16) || !aligned(c->v_scales, 16) ||
      !aligned(c->texp, 4))
    return fail(SNIP_E_ALIGN, "%s: the cache's buffers must be 16-byte aligned", who);
  int shift = 0;
  while ((1 << shift) < c->page_size) ++shift;
  *v = KvCache{static_cast<uint8_t*>(c->k_codes), static_cast<uint8_t*>(c->k_scales), static_cast<uint8_t*>(c->v_codes),
               static_cast<uint8_t*>(c->v_scales), c->format == SNIP_NVFP4 ? c->texp : nullptr, (int32_t)c->pages,
               c->kv_heads, shift};
  return SNIP_OK;
}

int check_batch(const char* who, const snipkv_batch* b, int64_t tokens, int page_size, KvBatch* v) {
  if (!b) return fail(SNIP_E_NULL, "%s: batch is NULL", who);
  if (!b->table || !b->lens) return fail(SNIP_E_NULL, "%s: table and lens must be non-NULL", who);
  if (!aligned(b->table, 4) || !aligned(b->lens, 4) || !aligned(b->cu, 4))
    return fail(SNIP_E_ALIGN, "%s: misaligned pointer", who);
  if (b->seqs < 1 || b->seqs > kMaxSeqs) return fail(SNIP_E_SHAPE, "%s: seqs=%lld outside 1 .. 2^20", who, (long long)b->seqs);
  if (b->max_pages < 1 || b->max_pages > kMaxLen / page_size)
    return fail(SNIP_E_SHAPE, "%s: max_pages=%lld outside 1 .. 2^30 / page_size", who, (long long)b->max_pages);
  if (b->table_ld < b->max_pages || b->table_ld > kMaxLd)
    return fail(SNIP_E_SHAPE, "%s: table_ld=%lld must be >= max_pages=%lld", who, (long long)b->table_ld,
                (long long)b->max_pages);
  if (tokens < 1 || tokens > kMaxTokens) return fail(SNIP_E_SHAPE, "%s: tokens=%lld outside 1 .. 2^20", who, (long long)tokens);
  if (!b->cu && tokens != b->seqs)
    return fail(SNIP_E_SHAPE, "%s: %lld tokens for %lld sequences need cu", who, (long long)tokens, (long long)b->seqs);
  *v = KvBatch{b->table, b->lens, b->cu, b->table_ld, (int32_t)(b->max_pages * page_size), (int32_t)b->seqs};
  return SNIP_OK;
}

int check_rows(const char* who, const char* name, const void* p, int type, int64_t ld, int64_t cols) {
  if (!p) return SNIP_OK;
  const int step = type == SNIPOP_F32 ? 4 : 8;
  if (ld < cols || ld > kMaxLd || ld % step)
    return fail(SNIP_E_SHAPE, "%s: %s: leading dimension %lld must be >= %lld and a multiple of %d", who, name,
                (long long)ld, (long long)cols, step);
  if (!aligned(p, 16)) return fail(SNIP_E_ALIGN, "%s: %s is not 16-byte aligned", who, name);
  return SNIP_OK;
}

int check_heads(const char* who, int64_t q_heads, int64_t kv_heads) {
  if (q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads)
    return fail(SNIP_E_SHAPE, "%s: q_heads=%lld must be a multiple of kv_heads=%lld up to %lld", who, (long long)q_heads,
                (long long)kv_heads, (long long)kMaxHeads);
  return SNIP_OK;
}

}  // namespace

extern "C" {

int snipkv_append(const void* q, int64_t ldq, int64_t q_heads, const void* k, int64_t ldk, const void* v, int64_t ldv,
                  int type, int64_t tokens, const float* cos, const float* sin, int64_t angles, int64_t rot_dim,
                  int interleaved, const int32_t* pos, const snipkv_cache* cache, const snipkv_batch* batch, void* q_out,
                  int64_t ldqo, void* stream) {
  const char* who = "snipkv_append";
  KvAppend a;
  std::memset(&a, 0, sizeof(a));
  int rc = check_cache(who, cache, &a.c);
  if (rc) return rc;
  if ((rc = check_batch(who, batch, tokens, cache->page_size, &a.b))) return rc;
  if (!q && !k) return fail(SNIP_E_NULL, "%s: neither queries nor keys given", who);
  if (!k != !v) return fail(SNIP_E_NULL, "%s: k and v must be given together", who);
  if (!q != !q_out) return fail(SNIP_E_NULL, "%s: q and q_out must be given together", who);
  if (type != SNIPOP_BF16 && type != SNIPOP_F32) return fail(SNIP_E_FORMAT, "%s: unknown element type %d", who, type);
  const int64_t D = cache->head_dim;
  if (!q) q_heads = 0;                                   // it may be anything then
  if (q && (rc = check_heads(who, q_heads, cache->kv_heads))) return rc;
  if ((rc = check_rows(who, "q", q, type, ldq, q_heads * D))) return rc;
  if ((rc = check_rows(who, "k", k, type, ldk, cache->kv_heads * D))) return rc;
  if ((rc = check_rows(who, "v", v, type, ldv, cache->kv_heads * D))) return rc;
  if ((rc = check_rows(who, "q_out", q_out, SNIPOP_BF16, ldqo, q_heads * D))) return rc;
  if (rot_dim < 0 || rot_dim > D || rot_dim % 64)
    return fail(SNIP_E_SHAPE, "%s: rot_dim=%lld must be a multiple of 64 up to head_dim=%lld", who, (long long)rot_dim,
                (long long)D);
  if (rot_dim) {
    if (!cos || !sin) return fail(SNIP_E_NULL, "%s: cos and sin must be non-NULL", who);
    if (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(pos, 4)) return fail(SNIP_E_ALIGN, "%s: misaligned pointer", who);
    if (angles < 1 || angles > (int64_t)1 << 40) return fail(SNIP_E_SHAPE, "%s: angles=%lld must be >= 1", who, (long long)angles);
  }
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.cos = cos;
  a.sin = sin;
  a.pos = pos;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldqo = ldqo;
  a.tokens = tokens;
  a.angles = angles;
  a.q_heads = (int32_t)q_heads;
  a.rot = (int32_t)rot_dim;
  a.interleaved = interleaved != 0;
  a.type = type;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double work = (double)tokens * (double)(q_heads + (k ? 2 * cache->kv_heads : 0)) * (double)D;
  const int slot = timing_begin(LaunchTag{SNIPKV_LAUNCH_APPEND, cache->format, -1, -1, work}, s);
  const hipError_t e = launch_kv_append(cache->format, cache->head_dim, a, s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "kv append launch"))) return rc;
  return ok();
}

int snipkv_gather(const snipkv_cache* cache, const snipkv_batch* batch, int64_t tokens, void* k, int64_t ldk, void* v,
                  int64_t ldv, void* stream) {
  const char* who = "snipkv_gather";
  KvGather a;
  std::memset(&a, 0, sizeof(a));
  int rc = check_cache(who, cache, &a.c);
  if (rc) return rc;
  if ((rc = check_batch(who, batch, tokens, cache->page_size, &a.b))) return rc;
  if (!k && !v) return fail(SNIP_E_NULL, "%s: no output given", who);
  const int64_t cols = (int64_t)cache->kv_heads * cache->head_dim;
  if ((rc = check_rows(who, "k", k, SNIPOP_BF16, ldk, cols))) return rc;
  if ((rc = check_rows(who, "v", v, SNIPOP_BF16, ldv, cols))) return rc;
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.ldk = ldk;
  a.ldv = ldv;
  a.tokens = tokens;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const double work = (double)tokens * (double)cols * ((k ? 1 : 0) + (v ? 1 : 0));
  const int slot = timing_begin(LaunchTag{SNIPKV_LAUNCH_APPEND, cache->format, -1, -1, work}, s);
  const hipError_t e = launch_kv_gather(cache->format, cache->head_dim, a, s);
  timing_end(slot, s);
  if ((rc = hip_check(e, "kv gather launch"))) return rc;
  return ok();
}

size_t snipkv_attn_workspace(int64_t tokens, int64_t seqs, int64_t q_heads, int64_t kv_heads, int64_t head_dim) {
  if (tokens < 1 || tokens > kMaxTokens || seqs < 1 || seqs > kMaxSeqs || kv_heads < 1 || kv_heads > kMaxHeads ||
      q_heads < 1 || q_heads > kMaxHeads || q_heads % kv_heads || !head_dim_ok(head_dim))
    return 0;
  const int64_t tiles = kv_attn_tiles(tokens, seqs, q_heads / kv_heads);
  if (tiles > kMaxTiles || tiles * kv_heads > (int64_t)1 << 30) return 0;      // steps are counted in 31 bits
  return align_up(kv_attn_slots((int)head_dim), kAlign);
}

int snipkv_attn(const void* q, int64_t ldq, int64_t q_heads, int64_t tokens, const snipkv_cache* cache,
                const snipkv_batch* batch, float scale, int64_t window, void* out, int64_t ldo, float* lse, void* ws,
                size_t ws_bytes, void* stream) {
  const char* who = "snipkv_attn";
  if (!q || !out) return fail(SNIP_E_NULL, "%s: q and out must be non-NULL", who);
  KvAttn a;
  std::memset(&a, 0, sizeof(a));
  int rc = check_cache(who, cache, &a.c);
  if (rc) return rc;
  if ((rc = check_batch(who, batch, tokens, cache->page_size, &a.b))) return rc;
  if ((rc = check_heads(who, q_heads, cache->kv_heads))) return rc;
  const int64_t cols = q_heads * cache->head_dim;
  if ((rc = check_rows(who, "q", q, SNIPOP_BF16, ldq, cols))) return rc;
  if ((rc = check_rows(who, "out", out, SNIPOP_BF16, ldo, cols))) return rc;
  const float scale2 = (float)((double)scale * 1.4426950408889634);   // of powers of two
  if (!(scale > 0.0f) || !std::isfinite(scale2)) return fail(SNIP_E_SHAPE, "%s: scale must be > 0 and up to 2e38", who);
  if (window < 0) return fail(SNIP_E_SHAPE, "%s: window=%lld must be >= 0", who, (long long)window);
  if (!aligned(lse, 4) || !aligned(ws, 16)) return fail(SNIP_E_ALIGN, "%s: misaligned pointer", who);
  const size_t need = snipkv_attn_workspace(tokens, batch->seqs, q_heads, cache->kv_heads, cache->head_dim);
  if (!need)
    return fail(SNIP_E_SHAPE, "%s: %lld tokens of %lld query heads a kv head are too many", who, (long long)tokens,
                (long long)(q_heads / cache->kv_heads));
  if (!ws || ws_bytes < need) return fail(SNIP_E_WORKSPACE, "%s: workspace of %zu bytes needed", who, need);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.part = static_cast<float*>(ws);
  a.ldq = ldq;
  a.ldo = ldo;
  a.tokens = tokens;
  a.q_heads = (int32_t)q_heads;
  a.group = (int32_t)(q_heads / cache->kv_heads);
  a.window = window <= INT32_MAX ? (int32_t)window : 0;    // positions are below that, lens being 32-bit
  a.scale = scale2;
  const KvPlan p = kv_attn_plan(cache->format, cache->head_dim, &a);
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto timed = [&](int kind, hipError_t (*launch)(int, int, const KvPlan&, const KvAttn&, hipStream_t)) {
    const int slot = timing_begin(LaunchTag{kind, cache->format, -1, -1, 4.0 * (double)tokens * (double)cols}, s);
    const hipError_t e = launch(cache->format, cache->head_dim, p, a, s);
    timing_end(slot, s);
    return hip_check(e, "kv attention launch");
  };
  if (p.prompt && (rc = timed(SNIPKV_LAUNCH_ATTN, launch_kv_prompt))) return rc;
  if (p.few && (rc = timed(SNIPKV_LAUNCH_ATTN, launch_kv_few))) return rc;
  if (p.join && (rc = timed(SNIPKV_LAUNCH_JOIN, launch_kv_join))) return rc;
  return ok();
}

}  // extern "C"
