// The 8-bit paged key/value cache: arguments and layout shared by the kernels
// that write it (kvcache.hip) and read it (kvcache.hip, attention.hip).
//
// One block holds the `page` tokens of one page and one head. A value is
// scale * (u - 128) with a byte u and the block's FP32 scale. The bytes of a
// block lie as the matrix instructions take them, so that a wave reads a tile
// with 16 consecutive bytes a lane and neither lanes nor LDS banks collide:
//   keys    [page/16][D/16][16 tokens][16 d]   (16 d of one token are one
//           lane's load: the MFMA contracts over d)
//   values  [page/4][D][4 tokens]              (4 d of four tokens are one
//           lane's load: the MFMA contracts over tokens)
#pragma once
#include "common.h"

namespace lowbit {

struct KvCache {
  uint8_t* k;
  uint8_t* v;
  float* ks;         // [pages][heads]
  float* vs;
  int64_t pages;
  int heads, page, D;
};

// The pages of the sequences: sequence b's tokens t lie in page
// table[b * width + t / page]; an entry outside 0 .. pages - 1 is no page
// (tokens there are neither written nor read).
struct KvTable {
  const int32_t* table;
  int64_t width;
  const int32_t* cu;      // [batch + 1] rows of the sequences in the dense operands
  const int32_t* start;   // [batch] first token (append, read) or length (attention)
  int64_t tokens;         // rows of the dense operands
  int batch, max_tokens;
};

struct KvRows {           // one dense operand [tokens][heads][D], last dimension of stride 1
  void* p;
  int64_t ts, hs;         // token and head stride, in elements
};

struct KvAppendArgs {
  KvCache c;
  KvTable t;
  KvRows k, v, q, qo;
  int q_heads, dtype, rot, inter;
  const float* cos;       // [rope_rows][rot / 2]
  const float* sin;
  int64_t rope_rows;
  int32_t* bad;           // nullable [2]: non-finite values, tokens without a place
  const void* k_norm;     // nullable [D] of norm_dtype: weights of the heads' norms
  const void* q_norm;
  int norm_dtype;
  float eps;
};

struct KvReadArgs {
  KvCache c;
  KvTable t;
  KvRows k, v;
  int dtype;
};

__device__ __forceinline__ int64_t k_byte(int t, int d, int D) {
  return (int64_t)(t >> 4) * 16 * D + (d >> 4) * 256 + (t & 15) * 16 + (d & 15);
}
__device__ __forceinline__ int64_t v_byte(int t, int d, int D) {
  return (int64_t)(t >> 2) * 4 * D + d * 4 + (t & 3);
}

// The rows [lo, hi) of the dense operands that belong to sequence b, kept
// inside [0, tokens) whatever the device array holds.
__device__ __forceinline__ void kv_rows(const KvTable& t, int b, int64_t* lo, int* n) {
  int64_t a = t.cu[b], e = t.cu[b + 1];
  a = a < 0 ? 0 : a > t.tokens ? t.tokens : a;
  e = e < a ? a : e > t.tokens ? t.tokens : e;
  *lo = a;
  *n = (int)(e - a < t.max_tokens ? e - a : t.max_tokens);
}

struct TurnArgs {         // norm and rotation of dense rows
  KvRows in[2], out[2];   // queries, keys
  int heads[2];           // 0: none
  const void* w[2];       // nullable
  int D, dtype, w_dtype, rot, inter;
  float eps;
  const float* cos;       // [rope_rows][rot / 2]
  const float* sin;
  int64_t rope_rows;
  const int32_t* pos;     // nullable [tokens]: else token t is at position t
  int64_t token0, tokens; // of this launch: token0 .. token0 + tokens - 1
  int32_t* bad;           // nullable [1]: tokens without a position
};

constexpr int kMaxPairs = 128;      // rot / 2
struct TableArgs {
  float* cos;             // [n][half]
  float* sin;
  int64_t n, first;
  int half;
  float magnitude;
  uint64_t turns[kMaxPairs];        // a position's angle in turns of 2^64
};

struct AttnArgs {
  KvCache c;
  KvTable t;              // start = tokens of each sequence in the cache, new ones included
  KvRows q, o;            // [tokens][q_heads][D]
  float* lse;             // nullable [tokens][q_heads]
  int q_heads, group;     // group = query heads per key/value head
  int dtype;
  float scale;            // times log2(e): the kernels work in powers of two
  int causal, window, max_len;
  int sinks;              // first tokens seen beside the window, 0 without one
  int splits, split_len;  // parts of the context, one workgroup each
  float* part;            // splits > 1: [splits][tokens * q_heads][D], then (max, sum) [splits][tokens * q_heads]
};

struct AttnPlan {
  bool few;               // 16-row tiles, else 32 rows a wave
  int waves;              // of a workgroup
  int splits, split_len;
};

enum AttnJoin { JOIN_NONE = 0, JOIN_BY_ROWS = 1, JOIN_BY_GROUPS = 2 };   // several rows a workgroup, or one

}  // namespace lowbit
