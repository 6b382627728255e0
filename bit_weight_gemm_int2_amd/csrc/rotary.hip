// Rotary positions apart from the cache: tables of cos and sin with the
// frequencies scaled for long contexts, and the norm of each head with the
// rotation of dense queries and keys.
#include <algorithm>

#include "kvcache.h"
#include "rotate.h"

namespace lowbit {

namespace {

// Tables: cos and sin of position * frequency. The angle is FP64, in quarter
// turns: whole quarters come off exactly, and the rest in [-1/2, 1/2] is rounded
// to FP32 once (an FP32 product at position 100000 would be off by thousandths of
// a turn). Its sine and cosine are their Taylor series to x^9 and x^10, which leave
// out less than 2e-9 at x = pi/4. Bound by the stores: a thread writes 16 bytes of
// each table, a wave whole kilobytes, past the caches.
__global__ __launch_bounds__(256) void tables_kernel(TableArgs g) {
  const int quads = g.half / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= g.n * quads) return;
  const int64_t p = i / quads;
  const int j = (int)(i - p * quads) * 4;
  const double pos = (double)(g.first + p);
  f32x4 c, s;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const double t = pos * g.quarters[j + e], q = __builtin_rint(t);
    const float x = (float)(t - q) * 1.57079632679489662f, y = x * x;
    const float a = __builtin_fmaf(x * y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, 1.0f / 362880, -1.0f / 5040),
                                                                           1.0f / 120), -1.0f / 6), x);
    const float b = __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, -1.0f / 3628800,
                                   1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const int k = (int)q;                                    // sine and cosine of x + k quarters
    const float u = k & 1 ? b : a, v = k & 1 ? a : b;
    s[e] = (k & 2 ? -u : u) * g.magnitude;
    c[e] = ((k + 1) & 2 ? -v : v) * g.magnitude;
  }
  __builtin_nontemporal_store(c, (f32x4*)(g.cos + p * g.half + j));
  __builtin_nontemporal_store(s, (f32x4*)(g.sin + p * g.half + j));
}

// Dense rows: thread = one unit of 16 values of a row (a token and head), rows
// in the order of tokens, then query heads, then key heads, so that a wave's
// loads lie together and a token's cos and sin stay in the L1.
template <int DT>
__global__ __launch_bounds__(256) void turn_kernel(TurnArgs g) {
  const int U = g.D / 16, shift = 31 - __builtin_clz(U);
  const uint32_t heads = g.heads[0] + g.heads[1];
  const uint32_t row = (blockIdx.x * 256u + threadIdx.x) >> shift;
  if (row >= (uint64_t)g.tokens * heads) return;
  const int u = threadIdx.x & (U - 1);
  const int64_t t = g.token0 + row / heads;
  int h = row % heads;
  const bool key = h >= g.heads[0];
  const bool counts = h == 0 && u == 0;
  h -= key ? g.heads[0] : 0;
  const KvRows& in = g.in[key];
  const KvRows& out = g.out[key];
  int d0, d1;
  unit_places(u, g.rot, g.inter, &d0, &d1);
  const int64_t to = t * out.ts + h * out.hs;
  const int64_t pos = g.pos ? (int64_t)g.pos[t] : t;
  float r[16];
  if (g.rot && (pos < 0 || pos >= g.rope_rows)) {
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] = 0.0f;
    if (g.bad && counts) atomicAdd(g.bad, 1);
  } else {
    const int64_t at = t * in.ts + h * in.hs;
    load8<DT, true>(in.p, at + d0, r);
    load8<DT, true>(in.p, at + d1, r + 8);
    Turn turn;
    load_turn(g.cos, g.sin, g.rot, u, pos, &turn);
    if (g.w[key]) {
      float w[16];
      load_weights(g.w[key], g.w_dtype, d0, d1, w);
      norm_unit(r, w, U, 1.0 / g.D, g.eps);
    }
    rotate_unit(r, turn, g.inter);
  }
  store8<DT>(out.p, to + d0, r);
  store8<DT>(out.p, to + d1, r + 8);
}

}  // namespace

hipError_t launch_rope_tables(const TableArgs& g, hipStream_t st) {
  // 2^31 threads a launch; a quad of 32 table rows at least in each
  const int64_t most = ((int64_t)1 << 31) / (g.half / 4);
  for (int64_t p = 0; p < g.n; p += most) {
    TableArgs a = g;
    a.first = g.first + p;
    a.n = std::min(most, g.n - p);
    a.cos = g.cos + p * g.half;
    a.sin = g.sin + p * g.half;
    tables_kernel<<<(unsigned)((a.n * (a.half / 4) + 255) / 256), 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

hipError_t launch_norm_rotate(const TurnArgs& g, hipStream_t st) {
  const int64_t units = (int64_t)(g.heads[0] + g.heads[1]) * (g.D / 16);   // of a token, at most 2^21
  const int64_t most = ((int64_t)1 << 31) / units;
  for (int64_t t = 0; t < g.tokens; t += most) {
    TurnArgs a = g;
    a.token0 = t;
    a.tokens = std::min(most, g.tokens - t);
    const unsigned blocks = (unsigned)((a.tokens * units + 255) / 256);
    if (g.dtype == DT_F16) turn_kernel<DT_F16><<<blocks, 256, 0, st>>>(a);
    else if (g.dtype == DT_BF16) turn_kernel<DT_BF16><<<blocks, 256, 0, st>>>(a);
    else turn_kernel<DT_F32><<<blocks, 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace lowbit
