// Writing and reading the 8-bit paged key/value cache (layout: kvcache.h).
//
// Append: key rows are rotated by their position (pairs (x, y) of the first
// `rot` dimensions become (x cos - y sin, x sin + y cos)), after the norm of
// the head where one is given; values are taken as they are. A block's scale is
// s = max(s_old, a / 127) with a the largest magnitude among the block's new
// values (s_old = 0 for a block that starts with this call), and a value r is stored as 128 + rint(r / s). When the
// scale grows, the block's older codes c follow it as rint(c s_old / s): each
// growth costs them at most half a step of the new scale. The quotients are
// real ones, so that ties (r = a / 2 is one) go to even: a bare product with
// 1 / s put one code in 10^4 of normal BF16 values a step off. One workgroup
// owns a block, so nothing is atomic and the result is a pure function of the
// input.
#include "kvcache.h"
#include "rotate.h"

namespace lowbit {

namespace {

constexpr int MAX_THREADS = 1024;
// scales below this are kept as 0 (reciprocals of scales stay finite); their values are
// below 2^-93 and become 0
constexpr float MIN_SCALE = 7.888609052210118e-31f;   // 2^-100

__device__ __forceinline__ uint32_t code(float r) {
  const float c = fminf(fmaxf(__builtin_rintf(r), -127.0f), 127.0f);
  return (uint32_t)(int)(c + 128.0f);
}

// four codes follow a grown scale (ratio = s_old / s)
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) o |= code(((float)((w >> (8 * i)) & 255u) - 128.0f) * ratio) << (8 * i);
  return o;
}

// max over the workgroup, in every thread
__device__ __forceinline__ float block_max(float x, float* lds) {
#pragma unroll
  for (int i = 32; i; i >>= 1) x = fmaxf(x, __shfl_xor(x, i));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  float m = lds[0];
  for (int i = 1; i < (int)blockDim.x / 64; ++i) m = fmaxf(m, lds[i]);
  return m;
}

struct Scale {
  float s, inv;           // the scale and its reciprocal (0 for a scale of 0: every quotient becomes 0)
};

// The block's new scale, and what its older codes are multiplied by.
__device__ __forceinline__ Scale new_scale(float top, float old, float* ratio) {
  float n = fmaxf(old, top / 127.0f);
  if (n < MIN_SCALE) n = 0.0f;
  *ratio = n > 0.0f ? old / n : 0.0f;
  return {n, n > 0.0f ? 1.0f / n : 0.0f};
}

// r / s: the product with the reciprocal and one correction by its exact
// remainder (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990). That is the quotient rounded once, but
// where it lies within 2^-21 of an FP32 step of a midpoint; an exact tie stays
// one. Full divisions took 69.1 us for 11000 tokens with their queries and the
// read-back, bare products 66.0, this 66.4.
__device__ __forceinline__ float quotient(float r, const Scale& s) {
  const float q = r * s.inv;
  return __builtin_fmaf(__builtin_fmaf(-q, s.s, r), s.inv, q);
}

__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const Scale& s) {
  return code(quotient(a, s)) | code(quotient(b, s)) << 8 | code(quotient(c, s)) << 16 | code(quotient(d, s)) << 24;
}

// Both writers read their new values once: the first KEEP units of a thread
// (all of them for blocks of 64 tokens of 128) stay in registers between the
// maximum and the codes; larger blocks read the rest again.
template <int DT, bool NORM>
__device__ void append_keys(const KvAppendArgs& g, int64_t row0, int64_t pos0, int p0, int n, int64_t id, int h,
                            float* lds, int* bad) {
  constexpr int KEEP = 2;
  const int D = g.c.D, U = D / 16;                           // a power of two
  uint8_t* block = g.c.k + (id * g.c.heads + h) * (int64_t)g.c.page * D;
  float* sp = g.c.ks + id * g.c.heads + h;
  const float old = p0 ? *sp : 0.0f;
  const int shift = 31 - __builtin_clz(U);
  const bool norm = NORM && g.k_norm != nullptr;
  float wk[16];                                              // a thread's units are all at one place of their rows
  if (norm) {
    int d0, d1;
    unit_places(threadIdx.x & (U - 1), g.rot, g.inter, &d0, &d1);
    load_weights(g.k_norm, g.norm_dtype, d0, d1, wk);
  }
  // unit i of the new rows, rotated; non-finite values are 0
  auto fetch = [&](int i, float* r) __attribute__((always_inline)) {
    const int t = i >> shift, u = i & (U - 1);
    int d0, d1;
    unit_places(u, g.rot, g.inter, &d0, &d1);
    const int64_t at = (row0 + t) * g.k.ts + h * g.k.hs;
    load8<DT>(g.k.p, at + d0, r);
    load8<DT>(g.k.p, at + d1, r + 8);
    Turn turn;
    load_turn(g.cos, g.sin, g.rot, u, pos0 + t, &turn);
    if (norm) norm_unit(r, wk, U, 1.0 / D, g.eps);
    rotate_unit(r, turn, g.inter);
    int count = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (!finite(r[e])) r[e] = 0.0f, ++count;
    return count;
  };
  auto store = [&](int i, const float* r, const Scale& s) __attribute__((always_inline)) {
    const int t = i >> shift, u = i & (U - 1);
    int d0, d1;
    unit_places(u, g.rot, g.inter, &d0, &d1);
    *(u32x2*)(block + k_byte(p0 + t, d0, D)) = u32x2{codes4(r[0], r[1], r[2], r[3], s), codes4(r[4], r[5], r[6], r[7], s)};
    *(u32x2*)(block + k_byte(p0 + t, d1, D)) = u32x2{codes4(r[8], r[9], r[10], r[11], s), codes4(r[12], r[13], r[14], r[15], s)};
  };
  float kept[KEEP][16], top = 0.0f;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < n * U) {
      *bad += fetch(i, kept[k]);
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(kept[k][e]));
    }
  }
  for (int i = threadIdx.x + KEEP * blockDim.x; i < n * U; i += blockDim.x) {
    float r[16];
    *bad += fetch(i, r);
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fabsf(r[e]));
  }
  float ratio;
  const Scale s = new_scale(block_max(top, lds), old, &ratio);
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < n * U) store(i, kept[k], s);
  }
  for (int i = threadIdx.x + KEEP * blockDim.x; i < n * U; i += blockDim.x) {
    float r[16];
    fetch(i, r);
    store(i, r, s);
  }
  if (p0 && s.s != old) {
    for (int i = threadIdx.x; i < p0 * U; i += blockDim.x) {
      u32x4* p = (u32x4*)(block + k_byte(i >> shift, (i & (U - 1)) * 16, D));
      u32x4 w = *p;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = rescale4(w[e], ratio);
      *p = w;
    }
  }
  if (threadIdx.x == 0) *sp = s.s;
}

// A unit here is four tokens (a quad of the block) by 8 dimensions.
template <int DT>
__device__ void append_values(const KvAppendArgs& g, int64_t row0, int p0, int n, int64_t id, int h, float* lds,
                              int* bad) {
  constexpr int KEEP = 1;
  const int D = g.c.D, F = D / 8;                            // a power of two
  uint8_t* block = g.c.v + (id * g.c.heads + h) * (int64_t)g.c.page * D;
  float* sp = g.c.vs + id * g.c.heads + h;
  const float old = p0 ? *sp : 0.0f;
  const int shift = 31 - __builtin_clz(F);
  const int q0 = p0 >> 2, q1 = (p0 + n + 3) >> 2, units = (q1 - q0) << shift;
  // the new values of unit i, 0 elsewhere and where not finite
  auto fetch = [&](int i, float (*r)[8]) __attribute__((always_inline)) {
    const int qd = q0 + (i >> shift), f = i & (F - 1);
    int count = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = 4 * qd + j - p0;
      if (t >= 0 && t < n) {
        load8<DT>(g.v.p, (row0 + t) * g.v.ts + h * g.v.hs + 8 * f, r[j]);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!finite(r[j][e])) r[j][e] = 0.0f, ++count;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[j][e] = 0.0f;
      }
    }
    return count;
  };
  Scale s;
  float ratio;
  auto store = [&](int i, float (*r)[8]) __attribute__((always_inline)) {
    const int qd = q0 + (i >> shift), f = i & (F - 1);
    const int first = p0 - 4 * qd, last = p0 + n - 4 * qd;   // new tokens first .. last - 1 of the quad
    const uint32_t older = first > 0 ? (1u << (8 * first)) - 1u : 0u;
    const uint32_t later = last < 4 ? ~((1u << (8 * last)) - 1u) : 0u;
    u32x4* p = (u32x4*)(block + v_byte(4 * qd, 8 * f, D));
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      u32x4 w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int d = 4 * half + e;
        w[e] = codes4(r[0][d], r[1][d], r[2][d], r[3][d], s);
      }
      if (older | later) {                                   // other tokens of the quad stay, older ones in the new scale
        const u32x4 was = p[half];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = (w[e] & ~(older | later)) | ((s.s != old ? rescale4(was[e], ratio) : was[e]) & older) | (was[e] & later);
      }
      p[half] = w;
    }
  };
  float kept[KEEP][4][8], top = 0.0f;
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < units) {
      *bad += fetch(i, kept[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(kept[k][j][e]));
    }
  }
  for (int i = threadIdx.x + KEEP * blockDim.x; i < units; i += blockDim.x) {
    float r[4][8];
    *bad += fetch(i, r);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(r[j][e]));
  }
  s = new_scale(block_max(top, lds), old, &ratio);
#pragma unroll
  for (int k = 0; k < KEEP; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    if (i < units) store(i, kept[k]);
  }
  for (int i = threadIdx.x + KEEP * blockDim.x; i < units; i += blockDim.x) {
    float r[4][8];
    fetch(i, r);
    store(i, r);
  }
  if (s.s != old) {                                          // quads of older tokens alone
    for (int i = threadIdx.x; i < q0 * (D / 4); i += blockDim.x) {
      u32x4* p = (u32x4*)block + i;
      u32x4 w = *p;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = rescale4(w[e], ratio);
      *p = w;
    }
  }
  if (threadIdx.x == 0) *sp = s.s;
}

// Rotate the queries of n tokens (heads first .. last - 1), the first
// `rotated` of which have a position; the others' become 0. A thread takes one
// unit of one token and walks the heads with its cos and sin in registers;
// with few tokens the heads are spread over threads too.
template <int DT, bool NORM>
__device__ void rotate_queries(const KvAppendArgs& g, int64_t row0, int64_t pos0, int n, int rotated, int first,
                               int last) {
  const int U = g.c.D / 16, shift = 31 - __builtin_clz(U), units = rotated << shift;
  const float zeros[8] = {};
  for (int i = threadIdx.x + units; i < n << shift; i += blockDim.x) {
    const int64_t to = (row0 + (i >> shift)) * g.qo.ts + 16 * (i & (U - 1));
    for (int h = first; h < last; ++h) {
      store8<DT>(g.qo.p, to + h * g.qo.hs, zeros);
      store8<DT>(g.qo.p, to + h * g.qo.hs + 8, zeros);
    }
  }
  if (!units) return;
  const int ways = max(1, min(last - first, (int)blockDim.x / units));
  const bool norm = NORM && g.q_norm != nullptr;
  float wq[16];
  if (norm) {
    int d0, d1;
    unit_places(threadIdx.x & (U - 1), g.rot, g.inter, &d0, &d1);
    load_weights(g.q_norm, g.norm_dtype, d0, d1, wq);
  }
  for (int i = threadIdx.x; i < units * ways; i += blockDim.x) {
    const int way = i / units, j = i - way * units, t = j >> shift, u = j & (U - 1);
    int d0, d1;
    unit_places(u, g.rot, g.inter, &d0, &d1);
    Turn turn;
    load_turn(g.cos, g.sin, g.rot, u, pos0 + t, &turn);
    const int64_t at = (row0 + t) * g.q.ts, to = (row0 + t) * g.qo.ts;
    if constexpr (NORM) {
      // two heads' loads before the first one's sum over lanes (11000 tokens with their queries: 64 us, one by one 69)
      for (int h = first + way; h < last; h += 2 * ways) {
        float r[2][16];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int64_t from = at + min(h + k * ways, last - 1) * g.q.hs;
          load8<DT, true>(g.q.p, from + d0, r[k]);
          load8<DT, true>(g.q.p, from + d1, r[k] + 8);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (h + k * ways >= last) break;
          if (norm) norm_unit(r[k], wq, U, 1.0 / g.c.D, g.eps);
          rotate_unit(r[k], turn, g.inter);
          store8<DT>(g.qo.p, to + (h + k * ways) * g.qo.hs + d0, r[k]);
          store8<DT>(g.qo.p, to + (h + k * ways) * g.qo.hs + d1, r[k] + 8);
        }
      }
    } else {
      for (int h = first + way; h < last; h += ways) {
        float r[16];
        load8<DT, true>(g.q.p, at + h * g.q.hs + d0, r);
        load8<DT, true>(g.q.p, at + h * g.q.hs + d1, r + 8);
        rotate_unit(r, turn, g.inter);
        store8<DT>(g.qo.p, to + h * g.qo.hs + d0, r);
        store8<DT>(g.qo.p, to + h * g.qo.hs + d1, r + 8);
      }
    }
  }
}

// grid: x = pages that a sequence's new tokens may touch, y = key heads,
// value heads, then groups of query heads, z = sequences. NORM: the norm of
// keys or queries, or both (a kernel of its own: without it the other's
// registers and results stay as they are).
template <int DT, bool NORM>
__global__ __launch_bounds__(MAX_THREADS) void append_kernel(KvAppendArgs g, int q_group) {
  __shared__ float lds[MAX_THREADS / 64];
  const int b = blockIdx.z, H = g.c.heads, page = g.c.page;
  int64_t row0;
  int n;
  kv_rows(g.t, b, &row0, &n);
  const int64_t start = max(g.t.start[b], 0);
  const int64_t slot = start / page + blockIdx.x;            // page of the sequence
  const int64_t first = max(start, slot * page), last = min(start + n, (slot + 1) * page);
  if (first >= last) return;
  row0 += first - start;
  n = (int)(last - first);
  const int role = blockIdx.y;
  int64_t known = last;                                      // positions that the tables cover
  if (g.rot && known > g.rope_rows) known = g.rope_rows;
  const int rotated = (int)max((int64_t)0, known - first);   // of the n tokens
  if (role >= 2 * H) {
    const int h0 = (role - 2 * H) * q_group;
    rotate_queries<DT, NORM>(g, row0, first, n, rotated, h0, min(g.q_heads, h0 + q_group));
    return;
  }
  const int64_t id = slot < g.t.width ? g.t.table[b * g.t.width + slot] : -1;
  if (id < 0 || id >= g.c.pages) {
    if (g.bad && role == 0 && threadIdx.x == 0) atomicAdd(g.bad + 1, n);
    return;
  }
  if (rotated < n && g.bad && role == 0 && threadIdx.x == 0) atomicAdd(g.bad + 1, n - rotated);
  if (!rotated) return;
  int bad = 0;
  const int p0 = (int)(first - slot * page);
  if (role < H) append_keys<DT, NORM>(g, row0, first, p0, rotated, id, role, lds, &bad);
  else append_values<DT>(g, row0, p0, rotated, id, role - H, lds, &bad);
  if (g.bad && bad) atomicAdd(g.bad, bad);
}

// The FP32 product as a value of its own: the compiler would fold a multiply
// into the conversion to FP16 (v_fma_mixlo_f16) and round the exact product
// once, which no other output type does.
__device__ __forceinline__ float value_of(float s, uint32_t u) {
  float r = s * ((float)u - 128.0f);
  asm("" : "+v"(r));
  return r;
}

// Dense rows of a range of the cache. grid as above: y = key heads, value heads
template <int DT>
__global__ __launch_bounds__(MAX_THREADS) void read_kernel(KvReadArgs g) {
  const int b = blockIdx.z, H = g.c.heads, page = g.c.page, D = g.c.D;
  int64_t row0;
  int n;
  kv_rows(g.t, b, &row0, &n);
  const int64_t start = max(g.t.start[b], 0);
  const int64_t slot = start / page + blockIdx.x;
  const int64_t first = max(start, slot * page), last = min(start + n, (slot + 1) * page);
  if (first >= last) return;
  row0 += first - start;
  n = (int)(last - first);
  const int p0 = (int)(first - slot * page);
  const bool values = (int)blockIdx.y >= H;
  const int h = blockIdx.y - (values ? H : 0);
  const int64_t id = slot < g.t.width ? g.t.table[b * g.t.width + slot] : -1;
  const bool there = id >= 0 && id < g.c.pages;
  const int64_t blk = there ? id * H + h : 0;
  const uint8_t* block = (values ? g.c.v : g.c.k) + blk * (int64_t)page * D;
  const float s = there ? (values ? g.c.vs : g.c.ks)[blk] : 0.0f;   // no page: zeros
  if (!values) {
    const int C = D / 8, shift = 31 - __builtin_clz(C);
    for (int i = threadIdx.x; i < n * C; i += blockDim.x) {
      const int t = i >> shift, d = (i & (C - 1)) * 8;
      const u32x2 w = *(const u32x2*)(block + k_byte(p0 + t, d, D));
      float r[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] = value_of(s, (w[e >> 2] >> (8 * (e & 3))) & 255u);
      store8<DT>(g.k.p, (row0 + t) * g.k.ts + h * g.k.hs + d, r);
    }
  } else {
    const int F = D / 8, shift = 31 - __builtin_clz(F), q0 = p0 >> 2, q1 = (p0 + n + 3) >> 2;
    for (int i = threadIdx.x; i < (q1 - q0) << shift; i += blockDim.x) {
      const int qd = q0 + (i >> shift), d = (i & (F - 1)) * 8;
      const u32x4* p = (const u32x4*)(block + v_byte(4 * qd, d, D));
      const u32x4 w0 = p[0], w1 = p[1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 4 * qd + j - p0;
        if (t < 0 || t >= n) continue;
        float r[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          r[e] = value_of(s, (w0[e] >> (8 * j)) & 255u);
          r[4 + e] = value_of(s, (w1[e] >> (8 * j)) & 255u);
        }
        store8<DT>(g.v.p, (row0 + t) * g.v.ts + h * g.v.hs + d, r);
      }
    }
  }
}

// pages that `tokens` consecutive tokens can touch, wherever they start
int page_slots(int tokens, int page) { return (int)(((int64_t)tokens + page - 2) / page + 1); }

}  // namespace

// Threads of a workgroup: one unit of 32 new values each of the two writers
// where the launch bound allows (128 tokens of 256 with 256 threads: 95 us
// for 3200 tokens of 4 heads with their queries, read back too, 67 with 1024).
static int block_threads(const KvTable& t, const KvCache& c) {
  const int64_t n = (int64_t)(t.max_tokens < c.page ? t.max_tokens : c.page) * c.D / 32;
  return (int)(n < 128 ? 128 : n > MAX_THREADS ? MAX_THREADS : (n + 63) / 64 * 64);
}

hipError_t launch_kv_append(const KvAppendArgs& g, hipStream_t st) {
  // two heads a workgroup: 66 us for 11000 tokens with read-back, 70 with four, 74 with eight
  const int q_group = 2;
  const dim3 grid(page_slots(g.t.max_tokens, g.c.page), 2 * g.c.heads + (g.q.p ? (g.q_heads + q_group - 1) / q_group : 0),
                  g.t.batch);
  const int threads = block_threads(g.t, g.c);
  if (g.k_norm || g.q_norm) {
    if (g.dtype == DT_F16) append_kernel<DT_F16, true><<<grid, threads, 0, st>>>(g, q_group);
    else if (g.dtype == DT_BF16) append_kernel<DT_BF16, true><<<grid, threads, 0, st>>>(g, q_group);
    else append_kernel<DT_F32, true><<<grid, threads, 0, st>>>(g, q_group);
  } else {
    if (g.dtype == DT_F16) append_kernel<DT_F16, false><<<grid, threads, 0, st>>>(g, q_group);
    else if (g.dtype == DT_BF16) append_kernel<DT_BF16, false><<<grid, threads, 0, st>>>(g, q_group);
    else append_kernel<DT_F32, false><<<grid, threads, 0, st>>>(g, q_group);
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& g, hipStream_t st) {
  const dim3 grid(page_slots(g.t.max_tokens, g.c.page), 2 * g.c.heads, g.t.batch);
  const int threads = block_threads(g.t, g.c);
  if (g.dtype == DT_F16) read_kernel<DT_F16><<<grid, threads, 0, st>>>(g);
  else if (g.dtype == DT_BF16) read_kernel<DT_BF16><<<grid, threads, 0, st>>>(g);
  else read_kernel<DT_F32><<<grid, threads, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace lowbit
