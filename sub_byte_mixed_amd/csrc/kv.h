// Internal launch interface between kv_api.hip and the kernels of the 4-bit
// key/value cache (kv_append.hip, kv_attn.hip), and what both know of its layout.
#pragma once

#include "../../include/snip_kv.h"
#include "kernels.h"

namespace snip {

struct KvCache {
  uint8_t *kc, *ks, *vc, *vs;
  const int32_t* texp;         // [2] or null (MXFP4)
  int32_t pages, heads;
  int32_t shift;               // log2 of the page's tokens
};

struct KvBatch {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;           // or null: row t is sequence t's only token
  int64_t table_ld;
  int32_t max_len;             // tokens that a sequence's table can name
  int32_t seqs;
};

struct KvAppend {
  KvCache c;
  KvBatch b;
  const void *q, *k, *v;       // q, or k and v, may be null
  uint16_t* q_out;
  const float *cos, *sin;
  const int32_t* pos;
  int64_t ldq, ldk, ldv, ldqo, tokens, angles;
  int32_t q_heads, rot, interleaved, type;
};

struct KvGather {
  KvCache c;
  KvBatch b;
  uint16_t *k, *v;             // one may be null
  int64_t ldk, ldv, tokens;
};

struct Left;                   // what the attention leaves for its second launch

struct KvAttn {
  KvCache c;
  KvBatch b;
  const uint16_t* q;
  uint16_t* out;
  float* lse;                  // or null
  float* part;                 // workspace of kv_attn_slots() bytes
  Left* left;                  // within it
  int64_t ldq, ldo, tokens;
  int32_t q_heads, group;      // query heads of a kv head
  int32_t window;              // 0: none
  int32_t split;               // the prompts among the sequences have a launch of their own: those
  int32_t few, some, far;      // of more rows than `few`, or than `some` with more keys than `far`
  int32_t step;                // keys of a step of work, a multiple of a workgroup's
  int32_t each;                // steps of a sequence where all have as many; 0: they follow from lens and cu
  float scale;                 // times log2 e
};

// Bytes of a key's piece, of its scales and of a value's piece.
constexpr int kv_key_piece(int dim) { return dim == 64 ? 8 : 16; }
constexpr int kv_value_piece(int dim) { return dim == 64 ? 2 : 4; }
constexpr int kv_scale_piece(int dim, int block) {
  return 2 * kv_key_piece(dim) / block ? 2 * kv_key_piece(dim) / block : 1;
}

// The launches of an attention call: prompts, few rows, and the joining of what
// the latter split.
struct KvPlan {
  bool prompt, few, join;
  bool two, wide, past;        // few rows: two row tiles; eight waves; read past the last-level cache
  int prompt_waves;            // of a workgroup for prompts
  unsigned prompt_wg, few_wg;  // workgroups
  int join_rows;
};

// Rows of a workgroup in the launch for prompts.
constexpr int kv_prompt_rows(int dim) { return dim == 256 ? 64 : 128; }

// Tiles of 16 rows of a call, a kv head's, at most; workspace bytes.
int64_t kv_attn_tiles(int64_t tokens, int64_t seqs, int64_t group);
size_t kv_attn_slots(int dim);
// Fills in what of `a` the plan decides (split, few, some, far, step, each, left).
KvPlan kv_attn_plan(int format, int dim, KvAttn* a);

hipError_t launch_kv_append(int format, int dim, const KvAppend& a, hipStream_t s);
hipError_t launch_kv_gather(int format, int dim, const KvGather& a, hipStream_t s);
hipError_t launch_kv_prompt(int format, int dim, const KvPlan& p, const KvAttn& a, hipStream_t s);
hipError_t launch_kv_few(int format, int dim, const KvPlan& p, const KvAttn& a, hipStream_t s);
hipError_t launch_kv_join(int format, int dim, const KvPlan& p, const KvAttn& a, hipStream_t s);

}  // namespace snip
