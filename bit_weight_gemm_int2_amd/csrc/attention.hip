// Attention of new queries over the 8-bit paged key/value cache (layout:
// kvcache.h): for a query at position i of its sequence and a head,
//   o = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q.k_j - max),
// over the cached tokens j that its mask leaves. k_j = s_k c_k(j) and
// v_j = s_v c_v(j) with one scale per page and head.
//
// Mathematics shared by the kernels:
//  * Codes are integers of at most 127 and exact in FP16: byte u becomes
//    0x6400 | u = 1024 + u by one byte permute for two codes, and a packed
//    add takes 1152 off. Queries are scaled by a power of two per row (exact)
//    so that BF16 ones keep their range, then rounded to FP16 (exact down to
//    2^-31 of the row's largest for BF16); every product is exact and sums are
//    FP32.
//  * The query's power of two and the softmax scale, then the key scales
//    multiply the FP32 scores. Value scales go into the softmax
//    exponent: with t_j = s_j + log2 s_v(j) (scores in powers of two) and the
//    running maximum m of t_j, p'_j = 2^(t_j - m) needs no scaling per page in
//    the values' product, and sum_j p_j is the FP32 sum of p'_j / s_v(j), taken
//    before p' is rounded to FP16 for the matrix product. One pass over the
//    cache, with the accumulators rescaled only when a maximum grows.
//  * FP16 probabilities: each is off by at most 2^-11, independently, so the
//    result by about 2^-12, less than a BF16 output's rounding (2^-9) and as
//    much as an FP16 one's; FP32 ones would double the matrix instructions.
//    They carry a factor of 2^TOP that puts the largest near the top of FP16's
//    range, so that tokens of 2^-28 of it (2^-23 for many rows) still have full
//    precision: where one token holds nearly all of the sum and has small
//    values, such tokens are the result (with the largest at 1, 4000 tokens of
//    2^-25 each beside such ones came out 32 to 48 % off).
//  * Scores are computed transposed (keys as the MFMA's rows), which leaves
//    every lane with probabilities of one query in just the order in which
//    the values' product wants them: no exchange between lanes but the
//    maximum.
//  * A page whose table entry is no page, and a token that the mask hides,
//    have t = -inf. A row that keeps nothing gives zeros (and lse = -inf).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "kvcache.h"

namespace lowbit {

namespace {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int PAGES = 264;                 // pages of one segment whose scales are held in LDS
constexpr float LN2 = 0.69314718055994530942f;
// Value scales below 2^-100 are those of all-zero blocks, whose tokens have
// weight and no value. They count as 2^-64: with the other scales between 2^-64
// and 2^40, neither p' / s_v of an equal score leaves FP32's range nor do the
// zeros push the others' p' below FP16's.
constexpr float MIN_SCALE = 0x1p-100f, ZERO_SCALE = 0x1p-64f;
constexpr float NEG_INF = -__builtin_inff();

struct Pages {
  int32_t blk[PAGES];                      // page * heads + head, 0 where there is no page
  float kf[PAGES], lv[PAGES], rv[PAGES];   // key scale, log2 and a unit's quotient of the value scale
};

// Two codes (bytes 0, 1 or 2, 3 of w) as FP16.
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel) {
  const uint32_t p = __builtin_amdgcn_perm(0x64646464u, w, sel);
  const f16x2 off = {(_Float16)-1152.0f, (_Float16)-1152.0f};
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2, p) + off);
}
__device__ __forceinline__ u32x4 codes8(uint32_t a, uint32_t b) {
  return u32x4{codes2(a, 0x04010400u), codes2(a, 0x04030402u), codes2(b, 0x04010400u), codes2(b, 0x04030402u)};
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const f16x2 h = {(_Float16)a, (_Float16)b};
  return __builtin_bit_cast(uint32_t, h);
}

// max / sum over the lanes that differ in bit 5 (32) or bits 4, 5 (16) of their
// number. A lane swap of x with a copy of itself leaves the two halves' values
// side by side. (The elements are taken as uint32_t first: a bit cast straight
// from an element of a vector reads element 0 whatever the index.)
__device__ __forceinline__ float max32(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  const uint32_t lo = r[0], hi = r[1];
  return fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi));
}
__device__ __forceinline__ float max16(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t lo = r[0], hi = r[1];
  return max32(fmaxf(__builtin_bit_cast(float, lo), __builtin_bit_cast(float, hi)));
}
__device__ __forceinline__ float sum32(float x) { return x + __shfl_xor(x, 32); }
__device__ __forceinline__ float sum16(float x) { return sum32(x + __shfl_xor(x, 16)); }

// What one row tile has to do: rows [row0, row0 + rows) of (token, head in
// group) pairs of one sequence and key/value head, tokens [t0, t1) of its
// context.
struct Work {
  int64_t lo;                              // first row of the sequence in the dense operands
  int n, rows, row0, len, t0, t1;
  __device__ __forceinline__ int pos(int row, int group) const { return len - n + row / group; }
};

__device__ __forceinline__ bool find_work(const AttnArgs& a, int b, int row0, int tile, int split, Work* w) {
  kv_rows(a.t, b, &w->lo, &w->n);
  w->rows = min(tile, w->n * a.group - row0);
  w->row0 = row0;
  if (w->rows <= 0) return false;
  const int64_t room = a.t.width * a.c.page;
  int len = max(0, min(a.t.start[b], a.max_len));
  w->len = len = (int)min((int64_t)len, room);
  const int last = w->pos(row0 + w->rows - 1, a.group), first = w->pos(row0, a.group);
  const int end = a.causal ? max(0, min(len, last + 1)) : len;
  const int beg = a.window ? max(0, first - a.window + 1) & ~15 : 0;
  w->t0 = (int)min((int64_t)end, beg + (int64_t)split * a.split_len);
  w->t1 = (int)min((int64_t)end, beg + ((int64_t)split + 1) * a.split_len);
  return true;
}

// Row (token row, head) of the dense operands for row r of the tile.
__device__ __forceinline__ void row_place(const AttnArgs& a, const Work& w, int h, int r, int64_t* token, int* head) {
  const int row = w.row0 + r;
  *token = w.lo + row / a.group;
  *head = h * a.group + row % a.group;
}

// The pages p0 .. p0 + np - 1 of sequence b: their blocks into LDS, then (by
// the same threads) the blocks' scales.
__device__ __forceinline__ void find_pages(const AttnArgs& a, int b, int h, int p0, int np, Pages* pg) {
  for (int i = threadIdx.x; i < np; i += blockDim.x) {
    const int32_t id = a.t.table[(int64_t)b * a.t.width + p0 + i];
    const bool there = id >= 0 && id < a.c.pages;
    pg->blk[i] = there ? id * a.c.heads + h : 0;
    pg->lv[i] = there ? 0.0f : NEG_INF;
  }
}
__device__ __forceinline__ void load_scales(const AttnArgs& a, int np, float unit, Pages* pg) {
  for (int i = threadIdx.x; i < np; i += blockDim.x) {
    const int32_t blk = pg->blk[i];
    const bool there = pg->lv[i] == 0.0f;
    const float ks = a.c.ks[blk], vs = a.c.vs[blk] >= MIN_SCALE ? a.c.vs[blk] : ZERO_SCALE;
    pg->kf[i] = there ? ks : 0.0f;
    pg->lv[i] = there ? __builtin_amdgcn_logf(vs) : NEG_INF;
    pg->rv[i] = unit / vs;
  }
}

// 8 values of a query as FP32
template <bool BF16>
__device__ __forceinline__ void values8(u32x4 w, float* x) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint16_t v = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    x[e] = BF16 ? bf16_bits_to_float(v) : half_bits_to_float(v);
  }
}

// The power of two that brings a row's largest magnitude into [2^14, 2^15), the
// top of FP16's range, and its inverse. Both stay normal numbers: a row below
// 2^-112 comes to lie lower (at 2^-7 with the smallest BF16 value), one with
// an infinity keeps it.
__device__ __forceinline__ void row_unit(float top, float* by, float* back) {
  const int e = min(max((int)(__builtin_bit_cast(uint32_t, top) >> 23), 15), 254);   // biased exponent; top >= 0
  *by = __builtin_bit_cast(float, (uint32_t)(268 - e) << 23);
  *back = __builtin_bit_cast(float, (uint32_t)(e - 14) << 23);
}

template <bool BF16>
__device__ __forceinline__ uint32_t out2(float x, float y) {
  return BF16 ? (uint32_t)float_to_bf16_bits(x) | (uint32_t)float_to_bf16_bits(y) << 16 : pack2(x, y);
}

__device__ __forceinline__ float inverse_sum(float l) { return l != 0.0f ? 1.0f / l : 0.0f; }

__device__ __forceinline__ void store_lse(const AttnArgs& a, int64_t token, int head, float m, float l) {
  if (a.lse) a.lse[token * a.q_heads + head] = l != 0.0f ? (m + __builtin_amdgcn_logf(l)) * LN2 : NEG_INF;
}

// ---------------------------------------------------------------------------
// Few rows (single tokens, drafts): 16 rows a workgroup, v_mfma_f32_16x16x32_f16.
// Bound by reading the cache where the GPU is full, by the conversion and the
// waves' latency (about 40 GB/s a CU, with 4, 8 or 16 waves alike) where not.
// Four waves walk 32-token steps of the part in turn, each with its own
// running maximum, and meet in LDS at the end. A wave reads its keys and values
// straight into registers (16 bytes a lane, whole kilobytes a wave); the next
// step's loads are in flight while one is computed. One token of 32 sequences
// over up to 8192 cached: 65 us, 4.7 TB/s.
// ---------------------------------------------------------------------------
// ONCE: one row tile a sequence and head, so the cache is read once, past the
// L2 (two sequences of 131072 tokens: 79 us against 90; with three row tiles
// 25 against 23).
template <bool BF16, int D, bool ONCE>
__global__ __launch_bounds__(256) void attend_few_kernel(AttnArgs a) {
  constexpr int NW = 4, NI = D / 64, LD = D + 4, STEP = 32 * NW;
  constexpr float TOP = 14.0f, UNSHIFT = 0x1p-14f;                     // p' up to 2^14
  __shared__ Pages pg;
  __shared__ float ml[NW][2][16];
  __shared__ __align__(16) float os[NW][16][LD];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int split = blockIdx.x, h = blockIdx.y % a.c.heads, b = blockIdx.z;
  Work w;
  if (!find_work(a, b, 16 * (blockIdx.y / a.c.heads), 16, split, &w)) return;
  const int shift = 31 - __builtin_clz(a.c.page);
  const int p0 = w.t0 >> shift;

  float m = NEG_INF, l = 0.0f;
  f32x4 o[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (w.t0 < w.t1) {
    const int last = (w.t1 - 1) & ~15;
    u32x4 kr[2][NI], vr[2][NI];
    auto load = [](const uint8_t* p) __attribute__((always_inline)) {
      return ONCE ? __builtin_nontemporal_load((const u32x4*)p) : *(const u32x4*)p;
    };
    auto load_k = [&](int j, int64_t at) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) kr[j][i] = load(a.c.k + at + lane * 16 + 1024 * i);
    };
    auto load_v = [&](int j, int64_t at) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) vr[j][i] = load(a.c.v + at + g * 4 * D + r * 16 + 256 * i);
    };
    // the 16-token tile at t (clamped into the part) of block blk
    auto tile_at = [&](int t, int32_t blk) __attribute__((always_inline)) {
      return ((int64_t)blk << shift) * D + (int64_t)(min(t, last) & (a.c.page - 1)) * D;
    };
    // the first step's tiles straight from the table: their loads and those of the scales are under way together
    int t = (w.t0 & ~15) + 32 * wave;
    if (t < w.t1) {
      int64_t at[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int32_t id = a.t.table[(int64_t)b * a.t.width + (min(t + 16 * j, last) >> shift)];
        at[j] = tile_at(t + 16 * j, id >= 0 && id < a.c.pages ? id * a.c.heads + h : 0);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) load_k(j, at[j]);
#pragma unroll
      for (int j = 0; j < 2; ++j) load_v(j, at[j]);
    }
    find_pages(a, b, h, p0, ((w.t1 - 1) >> shift) - p0 + 1, &pg);
    load_scales(a, ((w.t1 - 1) >> shift) - p0 + 1, 1.0f, &pg);
    // queries: lane (g, r) holds d = 16 (g + 4 i) + 8 half .. + 7 of row r
    int64_t token;
    int head;
    row_place(a, w, h, min(r, w.rows - 1), &token, &head);
    u32x4 qf[NI][2];
    float qs;
    {
      float x[NI][2][8], top = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          values8<BF16>(*(const u32x4*)((const uint16_t*)a.q.p + token * a.q.ts + head * a.q.hs + 16 * (g + 4 * i) + 8 * k), x[i][k]);
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[i][k][e]));
        }
      float by;
      row_unit(max16(top), &by, &qs);
      qs *= a.scale;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) qf[i][k][e] = pack2(x[i][k][2 * e] * by, x[i][k][2 * e + 1] * by);
    }
    const int pos = w.pos(w.row0 + min(r, w.rows - 1), a.group);
    const int hi = a.causal ? min(w.t1, pos + 1) : w.t1, lo = a.window ? pos - a.window + 1 : 0;
    // tokens that no row of the tile masks
    const int pos0 = w.pos(w.row0, a.group), pos1 = w.pos(w.row0 + w.rows - 1, a.group);
    const int all_hi = a.causal ? min(w.t1, pos0 + 1) : w.t1, all_lo = a.window ? pos1 - a.window + 1 : 0;
    __syncthreads();

    for (; t < w.t1; t += STEP) {
      f32x4 s[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        s[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            s[j] = mfma16<false>(codes8(kr[j][i][2 * k], kr[j][i][2 * k + 1]), qf[i][k], s[j]);
      }
      int64_t next[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) next[j] = tile_at(t + STEP + 16 * j, pg.blk[(min(t + STEP + 16 * j, last) >> shift) - p0]);
      if (t + STEP < w.t1) {
#pragma unroll
        for (int j = 0; j < 2; ++j) load_k(j, next[j]);
      }
      float rv[2], mx = NEG_INF;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int p = (min(t + 16 * j, last) >> shift) - p0;
        const float kf = pg.kf[p] * qs, lv = pg.lv[p];
        rv[j] = pg.rv[p];
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = __builtin_fmaf(s[j][e], kf, lv);
      }
      if (t < all_lo || t < w.t0 || t + 32 > all_hi) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = t + 16 * j + 4 * g + e;
            if (tok < lo || tok < w.t0 || tok >= hi) s[j][e] = NEG_INF;
          }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, s[j][e]);
      mx = max16(mx);
      if (__any(mx > m)) {
        const float n = fmaxf(m, mx), f = n > NEG_INF ? __builtin_amdgcn_exp2f(m - n) : 1.0f;
        m = n;
        l *= f;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i] *= f;
      }
      const float base = (m > NEG_INF ? m : 0.0f) - TOP;
      u32x4 pf;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = __builtin_amdgcn_exp2f(s[j][e] - base);
        l = __builtin_fmaf((p[0] + p[1]) + (p[2] + p[3]), rv[j], l);
        pf[2 * j] = pack2(p[0], p[1]);
        pf[2 * j + 1] = pack2(p[2], p[3]);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[4 * i + x] = mfma16<false>(codes8(vr[0][i][x], vr[1][i][x]), pf, o[4 * i + x]);
      if (t + STEP < w.t1) {
#pragma unroll
        for (int j = 0; j < 2; ++j) load_v(j, next[j]);
      }
    }
    l = sum16(l) * UNSHIFT;
  }
  // the waves meet: common maximum, then sums in wave order
  if (g == 0) {
    ml[wave][0][r] = m;
    ml[wave][1][r] = l;
  }
  __syncthreads();
  float top = ml[0][0][r];
#pragma unroll
  for (int k = 1; k < NW; ++k) top = fmaxf(top, ml[k][0][r]);
  const float f = top > NEG_INF ? __builtin_amdgcn_exp2f(m - top) * UNSHIFT : UNSHIFT;
  // lane (g, r): d = 64 i + 16 g + 4 e + x of row r
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *(f32x4*)&os[wave][r][64 * i + 16 * g + 4 * e] =
          f32x4{o[4 * i][e] * f, o[4 * i + 1][e] * f, o[4 * i + 2][e] * f, o[4 * i + 3][e] * f};
  __syncthreads();
  const int64_t total = a.t.tokens * a.q_heads;
  for (int i = tid; i < w.rows * (D / 4); i += 64 * NW) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    float mm = NEG_INF, ll = 0.0f;
#pragma unroll
    for (int k = 0; k < NW; ++k) mm = fmaxf(mm, ml[k][0][row]);
#pragma unroll
    for (int k = 0; k < NW; ++k)
      ll += ml[k][1][row] * (mm > NEG_INF ? __builtin_amdgcn_exp2f(ml[k][0][row] - mm) : 1.0f);
    f32x4 v = *(const f32x4*)&os[0][row][d];
#pragma unroll
    for (int k = 1; k < NW; ++k) v += *(const f32x4*)&os[k][row][d];
    int64_t token;
    int head;
    row_place(a, w, h, row, &token, &head);
    const int64_t slot = split * total + token * a.q_heads + head;
    if (a.splits == 1) {
      v *= inverse_sum(ll);
      *(u32x2*)((uint16_t*)a.o.p + token * a.o.ts + head * a.o.hs + d) = u32x2{out2<BF16>(v[0], v[1]), out2<BF16>(v[2], v[3])};
      if (d == 0) store_lse(a, token, head, mm, ll);
    } else {
      *(f32x4*)(a.part + slot * D + d) = v;
      if (d == 0) *(f32x2*)(a.part + a.splits * total * D + 2 * slot) = f32x2{mm, ll};
    }
  }
}

// ---------------------------------------------------------------------------
// Many rows (prompts): 128 or 256 rows a workgroup (32 a wave), tiles of 64
// tokens, v_mfma_f32_32x32x16_f16. Bound by the matrix and vector instructions
// (4096 queries over 20000 tokens: 1140 to 1190 us, 1.01 to 1.06 PFLOP/s).
// Codes go global -> registers two tiles ahead, are converted to FP16 once per
// workgroup one tile ahead and written to the other of two LDS stages in the
// order of the MFMA operands (16 consecutive bytes a lane both ways).
// ---------------------------------------------------------------------------
namespace many {
constexpr int TOK = 64;
// Powers of two that the running maximum may lag behind, and that p' is moved
// up by: together 15, FP16's limit. Rows ruled by tokens of value 0 were off by
// 0.0039 with 8 + 7, 0.0021 with 6 + 9, 0.0020 with 4 + 11 (0.0018 is the BF16
// output's rounding); four prompts of 512 took 24.1, 24.4 and 24.9 us.
constexpr float SLACK = 6.0f, TOP = 9.0f, UNSHIFT = 0x1p-9f;
template <int D> constexpr size_t stage() { return (size_t)TOK * D * 2 * 2; }
template <int D> constexpr size_t lds() { return 2 * stage<D>(); }
}  // namespace many

// The c-th run of 16 consecutive dimensions that a lane of half hh holds, and
// its first dimension. Value tile x has dimension 128 (x / 4) + 4 i + x % 4 in
// its row i (4 (i % 16) + x + 2 (i / 16) for 64 dimensions), and register e of
// a lane is row e % 4 + 8 (e / 4) + 4 hh.
template <int D>
__device__ __forceinline__ int many_run(const f32x16* o, int c, int hh, float* v) {
#pragma unroll
  for (int k = 0; k < 16; ++k)
    v[k] = D == 64 ? o[k & 1][(k >> 2) + 4 * c + 8 * ((k >> 1) & 1)] : o[4 * (c >> 2) + (k & 3)][4 * (c & 3) + (k >> 2)];
  return 128 * (c >> 2) + 4 * (8 * (c & 3) + 4 * hh);
}

template <bool BF16, int D, int W>
__global__ __launch_bounds__(64 * W, D == 256 ? W / 4 : 2) void attend_many_kernel(AttnArgs a) {
  constexpr int TOK = many::TOK, NT = 64 * W, ROWS = 32 * W;
  constexpr float SLACK = many::SLACK, TOP = many::TOP, UNSHIFT = many::UNSHIFT;
  // what a thread converts: NK pieces of KW words of a key, NV pieces of VW words of a pair of value quads
  constexpr int KW = TOK * D / 16 >= NT ? 4 : 2, NK = TOK * D / 4 / KW / NT;
  constexpr int VW = TOK * D / 32 >= NT ? 4 : TOK * D / 16 >= NT ? 2 : 1, NV = TOK * D / 8 / VW / NT;
  static_assert(NK >= 1 && NV >= 1, "every thread has a piece");
  constexpr int KB = TOK * D * 2;                                      // bytes of keys in a stage
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ Pages pg;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int hh = lane >> 5, r = lane & 31;
  // Workgroups go to the XCDs in turn, so with 8 heads an XCD keeps one head's
  // keys and values. Later row tiles see more of the context: the first
  // sequence begins with them, the next one ends with them, and so on.
  const int h = blockIdx.x % a.c.heads, split = blockIdx.x / a.c.heads, b = blockIdx.z;
  const int tile = b & 1 ? blockIdx.y : gridDim.y - 1 - blockIdx.y;
  Work w;
  if (!find_work(a, b, ROWS * tile, ROWS, split, &w)) return;
  const int shift = 31 - __builtin_clz(a.c.page);

  const int rr = min(32 * wave + r, w.rows - 1);
  int64_t token;
  int head;
  row_place(a, w, h, rr, &token, &head);
  u32x4 qf[D / 16];                                                    // the queries as they are, converted below
  float qs;
  {
    const int64_t at = token * a.q.ts + head * a.q.hs + 8 * hh;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) qf[s] = *(const u32x4*)((const uint16_t*)a.q.p + at + 16 * s);
  }
  auto convert_queries = [&]() __attribute__((always_inline)) {
    float x[8], top = 0.0f, by;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      values8<BF16>(qf[s], x);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[e]));
    }
    row_unit(max32(top), &by, &qs);
    qs *= a.scale;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      values8<BF16>(qf[s], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) qf[s][e] = pack2(x[2 * e] * by, x[2 * e + 1] * by);
    }
  };
  const int pos = w.pos(w.row0 + rr, a.group);
  const int hi = a.causal ? min(w.t1, pos + 1) : w.t1, lo = max(w.t0, a.window ? pos - a.window + 1 : 0);
  // tokens that no row of this wave masks
  const int f0 = min(32 * wave, w.rows - 1), f1 = min(32 * wave + 31, w.rows - 1);
  const int pos0 = w.pos(w.row0 + f0, a.group), pos1 = w.pos(w.row0 + f1, a.group);
  const int all_hi = a.causal ? min(w.t1, pos0 + 1) : w.t1, all_lo = max(w.t0, a.window ? pos1 - a.window + 1 : 0);
  // tokens that some row of this wave sees
  const int any_hi = 32 * wave >= w.rows ? 0 : a.causal ? min(w.t1, pos1 + 1) : w.t1, any_lo = max(w.t0, a.window ? pos0 - a.window + 1 : 0);

  float m = NEG_INF, l = 0.0f;
  f32x16 o[D / 32];
#pragma unroll
  for (int x = 0; x < D / 32; ++x)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[x][e] = 0.0f;

  uint32_t kr[NK][KW], vr[NV][2][VW];
  const int tbeg = w.t0 & ~15;
  const int seg_tokens = (PAGES - 8) << shift;                         // tokens whose pages fit the LDS
  for (int seg = tbeg; seg < w.t1; seg += seg_tokens) {                // a multiple of 64 tokens
    const int send = min(w.t1, seg + seg_tokens), p0 = seg >> shift, last = (send - 1) & ~15;
    const int np = ((send - 1) >> shift) - p0 + 1;
    if (seg != tbeg) __syncthreads();
    find_pages(a, b, h, p0, np, &pg);
    __syncthreads();
    auto tile_at = [&](int t) {                                        // bytes of the 16-token tile at t in its array
      t = min(t, last);
      return ((int64_t)pg.blk[(t >> shift) - p0] << shift) * D + (int64_t)(t & (a.c.page - 1)) * D;
    };
    auto words = [](uint32_t* to, const uint8_t* from, auto n) __attribute__((always_inline)) {
      constexpr int N = decltype(n)::value;
      if constexpr (N == 4) {
        const u32x4 w = *(const u32x4*)from;
        to[0] = w[0], to[1] = w[1], to[2] = w[2], to[3] = w[3];
      } else if constexpr (N == 2) {
        const u32x2 w = *(const u32x2*)from;
        to[0] = w[0], to[1] = w[1];
      } else {
        to[0] = *(const uint32_t*)from;
      }
    };
    auto fetch = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {                                   // word j of the keys' 16-token tiles
        const int j = (tid + NT * i) * KW, sub = j / (4 * D), in = j % (4 * D);
        words(kr[i], a.c.k + tile_at(t + 16 * sub) + in * 4, std::integral_constant<int, KW>());
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {                                   // (16-token tile, half, word): quads half and half + 2
        const int j = (tid + NT * i) * VW, sub = j / (2 * D), half = j / D % 2, d = j % D;
        const uint8_t* at = a.c.v + tile_at(t + 16 * sub) + half * 4 * D + d * 4;
        words(vr[i][0], at, std::integral_constant<int, VW>());
        words(vr[i][1], at + 8 * D, std::integral_constant<int, VW>());
      }
    };
    auto stage = [&](uint8_t* to) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {                                   // keys [32-token tile][d / 8][32 tokens][8 d]
        const int j = (tid + NT * i) * KW, sub = j / (4 * D), in = j % (4 * D) / 4, tk = 16 * (sub & 1) + (in & 15);
        uint8_t* at = to + (sub >> 1) * (32 * D * 2) + (2 * (in >> 4) + j % 4 / 2) * 512 + tk * 16;
#pragma unroll
        for (int e = 0; e < KW / 2; ++e) *(u32x4*)(at + 512 * e) = codes8(kr[i][2 * e], kr[i][2 * e + 1]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {                                   // values [16-token step][half][tile][32 rows][8 tokens]
        const int j = (tid + NT * i) * VW, sub = j / (2 * D), half = j / D % 2, f = j % D / 4;
        uint8_t* at = to + KB + (sub * 2 + half) * (D * 16);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const int y = j % 4 + e;
          const int x = D == 64 ? (y & 1) : 4 * (f >> 5) + y, row = D == 64 ? f + 16 * (y >> 1) : f & 31;
          *(u32x4*)(at + (x * 32 + row) * 16) = codes8(vr[i][0][e], vr[i][1][e]);
        }
      }
    };
    // Codes are fetched two tiles ahead and converted one tile ahead, between
    // the scores' matrix instructions; past the end the last tile repeats.
    fetch(seg);
    load_scales(a, np, UNSHIFT, &pg);                                  // the sum takes the factor off again
    if (seg == tbeg) convert_queries();
    stage(smem);
    fetch(seg + TOK);
    __syncthreads();
    int buf = 0;
    for (int t = seg; t < send; t += TOK, buf ^= 1) {
      const uint8_t* ks = smem + buf * many::stage<D>();
      const uint8_t* vs = ks + KB;
      uint8_t* const to = smem + (buf ^ 1) * many::stage<D>();
      if (t >= any_hi || t + TOK <= any_lo) {
        stage(to);
        fetch(t + 2 * TOK);
      } else {
        f32x16 s[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[j][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            s[j] = mfma32<false>(*(const u32x4*)(ks + j * (32 * D * 2) + (2 * k + hh) * 512 + r * 16), qf[k], s[j]);
        stage(to);
        fetch(t + 2 * TOK);
        // scores relative to m (to 0 before a row has seen anything), times 2^TOP
        const float base = m > NEG_INF ? m : 0.0f, low = base - TOP;
        float rv[4], mx = NEG_INF;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int p = (min(t + 16 * u, last) >> shift) - p0;
          const float kf = pg.kf[p] * qs, lv = pg.lv[p] - low;
          rv[u] = pg.rv[p];
#pragma unroll
          for (int e = 8 * (u & 1); e < 8 * (u & 1) + 8; ++e) s[u >> 1][e] = __builtin_fmaf(s[u >> 1][e], kf, lv);
        }
        if (t < all_lo || t + TOK > all_hi) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int tok = t + 32 * j + (e & 3) + 8 * (e >> 2) + 4 * hh;
              if (tok < lo || tok >= hi) s[j][e] = NEG_INF;
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e) mx = fmaxf(mx, s[j][e]);
        mx = max32(mx);
        // m follows the maximum only when that has grown by more than 2^SLACK: FP16 holds p' up to 2^(TOP + SLACK),
        // and the accumulators are seldom rescaled
        const bool move = mx > (m > NEG_INF ? TOP + SLACK : NEG_INF);
        if (__any(move)) {
          const float by = move ? mx - TOP : 0.0f, f = __builtin_amdgcn_exp2f(-by);
          if (move) m = base + by;
          // nothing accumulated yet: l and o are 0 and f may be anything finite
          const float g = fminf(f, 3.0e38f);
          l *= g;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) o[x] *= g;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[j][e] -= by;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(s[u >> 1][8 * (u & 1) + e]);
          l = __builtin_fmaf(((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7])), rv[u], l);
          const u32x4 pf = {pack2(p[0], p[1]), pack2(p[2], p[3]), pack2(p[4], p[5]), pack2(p[6], p[7])};
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            o[x] = mfma32<false>(*(const u32x4*)(vs + (u * 2 + hh) * (D * 16) + (x * 32 + r) * 16), pf, o[x]);
        }
      }
      __syncthreads();
    }
  }
  l = sum32(l);
  if (32 * wave + r >= w.rows) return;
  const int64_t total = a.t.tokens * a.q_heads, slot = split * total + token * a.q_heads + head;
  const float inv = a.splits == 1 ? inverse_sum(l) * UNSHIFT : UNSHIFT;
  if (hh == 0) {
    if (a.splits == 1) {
      store_lse(a, token, head, m, l);
    } else {
      float* p = a.part + a.splits * total * D + 2 * slot;
      p[0] = m;
      p[1] = l;
    }
  }
  // a lane holds runs of 16 dimensions of its row (many_run): two 16-byte stores each
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    float v[16];
    const int d = many_run<D>(o, c, hh, v);
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] *= inv;
    if (a.splits == 1) {
      uint16_t* to = (uint16_t*)a.o.p + token * a.o.ts + head * a.o.hs + d;
#pragma unroll
      for (int k = 0; k < 16; k += 8)
        *(u32x4*)(to + k) = u32x4{out2<BF16>(v[k], v[k + 1]), out2<BF16>(v[k + 2], v[k + 3]),
                                  out2<BF16>(v[k + 4], v[k + 5]), out2<BF16>(v[k + 6], v[k + 7])};
    } else {
#pragma unroll
      for (int k = 0; k < 16; k += 4) *(f32x4*)(a.part + slot * D + d + k) = f32x4{v[k], v[k + 1], v[k + 2], v[k + 3]};
    }
  }
}

// Join the parts of the context, one workgroup a row: the parts' weights meet
// in LDS, then groups of D / 4 threads take every (1024 / D)th part with four
// loads in flight, and their FP32 sums are added in group order.
// Latency-bound (three dependent reads): 32 parts of 80 rows of 128 take 4.6 us,
// one wave a row walking the parts in turn took 37 us.
template <bool BF16, int D>
__global__ __launch_bounds__(256) void attend_join_kernel(AttnArgs a) {
  constexpr int TPR = D / 4, NG = 256 / TPR, CH = 256;                 // threads a part, parts at a time, weights held
  __shared__ float wt[CH], red[2][4];
  __shared__ __align__(16) f32x4 acc[NG][TPR];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t total = a.t.tokens * a.q_heads, row = blockIdx.x + (int64_t)blockIdx.y * gridDim.x;
  if (row >= total) return;
  const f32x2* ml = (const f32x2*)(a.part + a.splits * total * D);
  float m = NEG_INF;
  for (int s = tid; s < a.splits; s += 256) m = fmaxf(m, ml[s * total + row][0]);
#pragma unroll
  for (int i = 32; i; i >>= 1) m = fmaxf(m, __shfl_xor(m, i));
  if (lane == 0) red[0][wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  const float base = m > NEG_INF ? m : 0.0f;
  const int gr = tid / TPR, d = tid % TPR * 4;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  float l = 0.0f;
  for (int c0 = 0; c0 < a.splits; c0 += CH) {
    const int nc = min(CH, a.splits - c0);
    if (c0) __syncthreads();
    if (tid < nc) {
      const f32x2 x = ml[(c0 + tid) * total + row];
      // a part that saw nothing has a sum of 0: weight 0 and nothing to read
      const float f = x[1] != 0.0f ? __builtin_amdgcn_exp2f(x[0] - base) : 0.0f;
      wt[tid] = x[1] != 0.0f ? f : -1.0f;
      l += x[1] != 0.0f ? x[1] * f : 0.0f;
    }
    __syncthreads();
    for (int s = gr; s < nc; s += 4 * NG) {
      f32x4 p[4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = s + u * NG;
        f[u] = k < nc ? wt[k] : -1.0f;
        p[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (!(f[u] < 0.0f)) p[u] = *(const f32x4*)(a.part + ((c0 + k) * total + row) * D + d);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (!(f[u] < 0.0f)) v += f[u] * p[u];
    }
  }
  acc[gr][tid % TPR] = v;
#pragma unroll
  for (int i = 32; i; i >>= 1) l += __shfl_xor(l, i);
  if (lane == 0) red[1][wave] = l;
  __syncthreads();
  if (gr) return;
  l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
#pragma unroll
  for (int k = 1; k < NG; ++k) v += acc[k][tid];
  v *= inverse_sum(l);
  const int64_t token = row / a.q_heads;
  if (token < a.t.cu[0] || token >= a.t.cu[a.t.batch]) return;         // no sequence's: no part was written
  const int head = (int)(row % a.q_heads);
  *(u32x2*)((uint16_t*)a.o.p + token * a.o.ts + head * a.o.hs + d) = u32x2{out2<BF16>(v[0], v[1]), out2<BF16>(v[2], v[3])};
  if (tid == 0) store_lse(a, token, head, m, l);
}

constexpr int FEW_ROWS = 80;
constexpr int FEW_SPLIT = 4096;            // tokens of a part that PAGES covers at pages of 16 (plus one page of offset)

template <bool BF16, int D, int W>
void launch_many(const AttnArgs& a, int rows, hipStream_t st) {
  attend_many_kernel<BF16, D, W><<<dim3(a.c.heads * a.splits, (rows + 32 * W - 1) / (32 * W), a.t.batch), 64 * W,
                                   many::lds<D>(), st>>>(a);
}

template <bool BF16, int D>
hipError_t launch(const AttnArgs& a, AttnPlan p, hipStream_t st) {
  const int rows = a.t.max_tokens * a.group;
  if (p.few && rows <= 16)
    attend_few_kernel<BF16, D, true><<<dim3(a.splits, a.c.heads, a.t.batch), 256, 0, st>>>(a);
  else if (p.few)
    attend_few_kernel<BF16, D, false><<<dim3(a.splits, a.c.heads * ((rows + 15) / 16), a.t.batch), 256, 0, st>>>(a);
  else if (p.waves == 4)
    launch_many<BF16, D, 4>(a, rows, st);
  else if constexpr (D == 128)
    launch_many<BF16, D, 8>(a, rows, st);
  if (a.splits > 1) {
    const int64_t total = a.t.tokens * a.q_heads, nx = std::min<int64_t>(total, 1 << 22);   // nx * 256 threads fit 32 bits
    attend_join_kernel<BF16, D><<<dim3((unsigned)nx, (unsigned)((total + nx - 1) / nx)), 256, 0, st>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

// Which kernel, how many waves a workgroup, and how many parts the context is
// split into. Up to 80 rows go in tiles of 16, each reading the context again
// from the caches (16 sequences of up to 6000 tokens with 40 rows: 26 us
// against 36 in a tile of 128 rows; 68 rows, four sequences: 23 against 36).
// For them the number of parts that a rough time estimate likes best: a round
// of workgroups costs about 2 us and, a step of 128 tokens, 0.8 us or its
// bytes at 40 GB/s a CU or, for lengths 0.6 of the longest, 5 TB/s; a join,
// with its launch, 6 us and 0.02 a part (one sequence of 1000 tokens and 8
// heads: 9.2 us in 7 parts against 10.2 whole on the GPU, 16.3 against 12.6
// from Python; 8 of 2000: 13.2 in parts, 16.2 whole). But at least enough
// parts of 1024 tokens to fill the GPU, since lengths are ragged.
// Many rows: parts until the row tiles fill the GPU twice.
AttnPlan attention_plan(int64_t batch, int heads, int group, int64_t max_tokens, int64_t max_len, int window, int D,
                        int num_cu) {
  const int64_t rows = max_tokens * group;
  AttnPlan p{};
  p.few = rows <= FEW_ROWS;
  int64_t span = max_len;
  if (window) span = std::min(span, (int64_t)window + max_tokens + 16);
  int64_t n = 1, len;
  if (p.few) {
    p.waves = 4;
    const int64_t tiles = batch * heads * ((rows + 15) / 16);
    const int64_t slots = (int64_t)num_cu * (D == 256 ? 2 : D == 128 ? 4 : 6);   // resident workgroups
    const int64_t fill = std::min(slots / std::max<int64_t>(tiles, 1), span / 1024);
    const int64_t least = std::max<int64_t>(1, (span + FEW_SPLIT - 1) / FEW_SPLIT);
    double best = 1e30;
    for (int64_t k = least; k == least || (k <= 768 && k * 128 <= span); k += k < 4 ? 1 : k / 3) {
      const int64_t steps = (span + 128 * k - 1) / (128 * k), rounds = (tiles * k + slots - 1) / slots;
      const double wgs = (double)std::min(tiles * k, slots), bytes = 256.0 * D;
      const double step = std::max({0.8, std::ceil(wgs / num_cu) * bytes / 4.0e4, 0.6 * wgs * bytes / 5.0e6});
      const double us = rounds * (2.0 + step * steps) + (k > 1 ? 6.0 + 0.02 * k : 0.0);
      if (us < best) {
        best = us;
        n = k;
      }
    }
    n = std::max(n, fill);
    len = std::min<int64_t>((span + n - 1) / n, FEW_SPLIT);
  } else {
    // 256 rows a workgroup halve the conversion of codes per row but leave one
    // workgroup a CU: only where its tiles are long and fill two rounds (32
    // query heads, 4000 queries over 20000 tokens, 504 tiles: 1127 us against
    // 1217 with 128 rows; 5000, 632 tiles: 1539 against 1491; 3000, 376 tiles:
    // 1045 against 970; one round would do as well, 2000, 250 tiles: 616
    // against 660; shorter contexts gain nothing, two of 4000 over 5000: 330
    // against 332)
    p.waves = D == 128 && span >= 8192 && batch * heads * ((rows + 255) / 256) >= 2 * num_cu ? 8 : 4;
    const int64_t tiles = batch * heads * ((rows + 32 * p.waves - 1) / (32 * p.waves));
    n = std::max<int64_t>(1, std::min((int64_t)8 * num_cu / p.waves / std::max<int64_t>(tiles, 1), span / 1024));
    len = (span + n - 1) / n;
  }
  len = std::max<int64_t>(128, (len + 127) / 128 * 128);
  p.split_len = (int)std::min<int64_t>(len, (int64_t)1 << 30);
  p.splits = (int)std::max<int64_t>(1, (span + len - 1) / len);
  return p;
}

hipError_t launch_attention(const AttnArgs& a, AttnPlan p, hipStream_t st) {
  const bool bf = a.dtype == DT_BF16;
  if (a.c.D == 64) return bf ? launch<true, 64>(a, p, st) : launch<false, 64>(a, p, st);
  if (a.c.D == 128) return bf ? launch<true, 128>(a, p, st) : launch<false, 128>(a, p, st);
  return bf ? launch<true, 256>(a, p, st) : launch<false, 256>(a, p, st);
}

}  // namespace lowbit
