// Rotary positions apart from the cache: tables of cos and sin with the
// frequencies scaled for long contexts, and the norm of each head with the
// rotation of dense queries and keys.
#include <algorithm>

#include "kvcache.h"
#include "rotate.h"

namespace lowbit {

namespace {

// Tables: cos and sin of position * frequency. An angle is a fraction of a turn in
// 64 bits of fixed point, so that whole turns fall off by themselves and the next
// position is one addition (an FP32 product at position 100000 would be off by
// thousandths of a turn). The nearest quarter turn comes off its upper half, and
// the rest, at most 1/8 turn to 2^-32, becomes FP32. Its sine and cosine are their
// Taylor series to x^9 and x^10, which leave out less than 2e-9 at x = pi/4. FP32
// there is a choice: entries are up to 1.2e-7 off (1.4 times the RMS error of the
// 64-bit value rounded once, up to 5.2e-8), a quarter of the contract's 2^-21. A
// thread writes 16 bytes of each table for ROWS positions, a wave whole kilobytes,
// past the caches; bound by the stores (131072 positions of 64 pairs: 12.3 to 12.9
// us, 5.2 to 5.5 TB/s; an earlier form of 13.6 us took 14.8, 13.8 and 13.9 with 1, 4
// or 8 positions a thread).
constexpr int ROWS = 2;

__global__ __launch_bounds__(256) void tables_kernel(TableArgs g) {
  const int quads = g.half / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t p = i / quads * ROWS;
  if (p >= g.n) return;
  const int j = (int)(i % quads) * 4;
  uint64_t angle[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) angle[e] = (uint64_t)(g.first + p) * g.turns[j + e];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (p + k >= g.n) return;
    f32x4 c, s;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t t = (uint32_t)(angle[e] >> 32) + 0x20000000u;
      const uint32_t q = t >> 30;                            // sine and cosine of x + q quarters
      const float x = (float)((int)(t & 0x3fffffffu) - 0x20000000) * (1.57079632679489662f / 0x40000000), y = x * x;
      const float a = __builtin_fmaf(x * y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, 1.0f / 362880, -1.0f / 5040),
                                                                             1.0f / 120), -1.0f / 6), x);
      const float b = __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, __builtin_fmaf(y, -1.0f / 3628800,
                                     1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
      const float u = q & 1 ? b : a, v = q & 1 ? a : b;
      s[e] = (q & 2 ? -u : u) * g.magnitude;
      c[e] = ((q + 1) & 2 ? -v : v) * g.magnitude;
      angle[e] += g.turns[j + e];
    }
    __builtin_nontemporal_store(c, (f32x4*)(g.cos + (p + k) * g.half + j));
    __builtin_nontemporal_store(s, (f32x4*)(g.sin + (p + k) * g.half + j));
  }
}

// Dense rows: thread = 16 values of a row (a token and head) in two pieces of 8,
// rows in the order of tokens, then query heads, then key heads, so that a wave's
// loads lie together and a token's cos and sin stay in the L1. Pieces are placed
// so that a rotated pair never leaves a thread and neighbouring lanes take
// neighbouring 16 bytes: with halves apart (d, d + rot / 2) one piece in each
// half of the rotated part, or of the rest; with neighbours paired one in each
// half of the row. Bound by memory; every load is issued before the first is
// waited for, so there are no branches around them: places that are not there
// are read at one that is. 4608 tokens of 24 + 24 heads of 128: 24.6 us, 4.7 TB/s
// (with branches, the sum through the LDS and 32 bytes a lane 29.1).
// W: the type of the norms' weights, DT_NONE without norms.
template <int DT, int W, bool INTER>
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
  const uint8_t* in = (const uint8_t*)(key ? g.in[1].p : g.in[0].p);
  const int32_t listed = *(g.pos ? g.pos + t : (const int32_t*)in);
  const int64_t pos = g.pos ? (int64_t)listed : t;
  const bool there = !g.rot || (pos >= 0 && pos < g.rope_rows);
  const int half = g.rot / 2;
  const bool turned = 16 * u < g.rot;
  const int rest = g.rot + 8 * u - half;                       // past the rotated part
  const int d0 = INTER || turned ? 8 * u : rest;
  const int d1 = INTER ? g.D / 2 + 8 * u : turned ? half + 8 * u : rest + (g.D - g.rot) / 2;
  const bool on0 = INTER ? d0 < g.rot : turned, on1 = INTER ? d1 < g.rot : turned;
  const int64_t at = t * (key ? g.in[1].ts : g.in[0].ts) + h * (key ? g.in[1].hs : g.in[0].hs);
  float r[16], w[16], c[8], s[8];
  load8<DT, true>(in, at + d0, r);
  load8<DT, true>(in, at + d1, r + 8);
  if constexpr (W != DT_NONE) {
    const void* own = key ? g.w[1] : g.w[0];
    const void* from = own ? own : key ? g.w[0] : g.w[1];
    load8<W>(from, d0, w);
    load8<W>(from, d1, w + 8);
  }
  if (g.rot) {
    // pairs of the first piece, then of the second; with halves apart the pieces share all eight
    const int64_t line = there ? pos * half : 0;
    const int p0 = INTER ? (on0 ? d0 / 2 : 0) : on0 ? d0 : 0, p1 = INTER ? (on1 ? d1 / 2 : 0) : p0 + 4;
    load4(g.cos + line + p0, c);
    load4(g.cos + line + p1, c + 4);
    load4(g.sin + line + p0, s);
    load4(g.sin + line + p1, s + 4);
  }
  if constexpr (W != DT_NONE) {
    const bool norm = key ? g.w[1] != nullptr : g.w[0] != nullptr;
    const float by = norm_factor(r, norm, U, 1.0 / g.D, g.eps);
#pragma unroll
    for (int e = 0; e < 16; ++e) r[e] = norm ? r[e] * by * w[e] : r[e];
  }
  if (g.rot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : i + 8;
      const bool on = i < 4 ? on0 : on1;
      const float x = r[a], y = r[b];
      r[a] = on ? __builtin_fmaf(x, c[i], -(y * s[i])) : x;
      r[b] = on ? __builtin_fmaf(x, s[i], y * c[i]) : y;
    }
    if (!there) {
#pragma unroll
      for (int e = 0; e < 16; ++e) r[e] = 0.0f;
      if (g.bad && counts) atomicAdd(g.bad, 1);
    }
  }
  void* out = key ? g.out[1].p : g.out[0].p;
  const int64_t to = t * (key ? g.out[1].ts : g.out[0].ts) + h * (key ? g.out[1].hs : g.out[0].hs);
  store8<DT>(out, to + d0, r);
  store8<DT>(out, to + d1, r + 8);
}

template <int DT, int W>
void launch_turn(const TurnArgs& a, unsigned blocks, hipStream_t st) {
  if (a.inter) turn_kernel<DT, W, true><<<blocks, 256, 0, st>>>(a);
  else turn_kernel<DT, W, false><<<blocks, 256, 0, st>>>(a);
}

template <int DT>
void launch_turn(const TurnArgs& a, unsigned blocks, hipStream_t st) {
  if (a.w_dtype == DT_NONE) launch_turn<DT, DT_NONE>(a, blocks, st);
  else if (a.w_dtype == DT_F16) launch_turn<DT, DT_F16>(a, blocks, st);
  else if (a.w_dtype == DT_BF16) launch_turn<DT, DT_BF16>(a, blocks, st);
  else launch_turn<DT, DT_F32>(a, blocks, st);
}

}  // namespace

hipError_t launch_rope_tables(const TableArgs& g, hipStream_t st) {
  const int64_t most = ((int64_t)1 << 31) / (g.half / 4);   // positions of a launch, at least 2^26
  for (int64_t p = 0; p < g.n; p += most) {
    TableArgs a = g;
    a.first = g.first + p;
    a.n = std::min(most, g.n - p);
    a.cos = g.cos + p * g.half;
    a.sin = g.sin + p * g.half;
    const int64_t threads = (a.n + ROWS - 1) / ROWS * (a.half / 4);
    tables_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, st>>>(a);
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
    if (g.dtype == DT_F16) launch_turn<DT_F16>(a, blocks, st);
    else if (g.dtype == DT_BF16) launch_turn<DT_BF16>(a, blocks, st);
    else launch_turn<DT_F32>(a, blocks, st);
  }
  return hipGetLastError();
}

}  // namespace lowbit
