// Writing and reading the 8-bit paged key/value cache (layout: kvcache.h).
//
// Append: key rows are rotated by their position (pairs (x, y) of the first
// `rot` dimensions become (x cos - y sin, x sin + y cos)), values are taken as
// they are. A block's scale is s = max(s_old, a / 127) with a the largest
// magnitude among the block's new values (s_old = 0 for a block that starts
// with this call), and a value r is stored as 128 + rint(r / s). When the
// scale grows, the block's older codes c follow it as rint(c s_old / s): each
// growth costs them at most half a step of the new scale. One workgroup owns
// a block, so nothing is atomic and the result is a pure function of the
// input.
#include "kvcache.h"

namespace lowbit {

namespace {

constexpr int APPEND_THREADS = 256;
// scales below this are kept as 0 (1 / s must stay finite); their values are
// below 2^-93 and become 0
constexpr float MIN_SCALE = 7.888609052210118e-31f;   // 2^-100

template <int DT>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (DT == DT_F16) return half_bits_to_float(((const uint16_t*)p)[i]);
  if constexpr (DT == DT_BF16) return bf16_bits_to_float(((const uint16_t*)p)[i]);
  return ((const float*)p)[i];
}

// N consecutive values (16-byte aligned in memory for N = 16 and for FP32; 8 bytes for N = 4 of 16 bits)
template <int DT, int N>
__device__ __forceinline__ void load_row(const void* p, int64_t i, float* r) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const f32x4 w = *(const f32x4*)((const float*)p + i + 4 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) r[4 * j + e] = w[e];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      const u32x2 w = *(const u32x2*)((const uint16_t*)p + i + 4 * j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint16_t h = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
        r[4 * j + e] = DT == DT_F16 ? half_bits_to_float(h) : bf16_bits_to_float(h);
      }
    }
  }
}

template <int DT, int N>
__device__ __forceinline__ void store_row(void* p, int64_t i, const float* r) {
  if constexpr (DT == DT_F32) {
#pragma unroll
    for (int j = 0; j < N / 4; ++j)
      *(f32x4*)((float*)p + i + 4 * j) = f32x4{r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]};
  } else {
#pragma unroll
    for (int j = 0; j < N / 4; ++j) {
      u32x2 w;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = r[4 * j + 2 * e], y = r[4 * j + 2 * e + 1];
        w[e] = DT == DT_F16 ? (uint32_t)float_to_half_bits(x) | (uint32_t)float_to_half_bits(y) << 16
                            : (uint32_t)float_to_bf16_bits(x) | (uint32_t)float_to_bf16_bits(y) << 16;
      }
      *(u32x2*)((uint16_t*)p + i + 4 * j) = w;
    }
  }
}

// Unit u of a row is 32 values in two pieces of 16, placed so that a rotated
// pair never leaves a unit: with halves apart ("x, y" = d, d + rot / 2) the
// pieces are 16 u and rot / 2 + 16 u, with neighbours paired (and past the
// rotated part) they are 32 u and 32 u + 16.
__device__ __forceinline__ void unit_places(int u, int rot, int inter, int* d0, int* d1) {
  if (!inter && 32 * u < rot) {
    *d0 = 16 * u;
    *d1 = rot / 2 + 16 * u;
  } else {
    *d0 = 32 * u;
    *d1 = 32 * u + 16;
  }
}

// Rotate one unit: a holds the values of its first piece, b of its second.
__device__ __forceinline__ void rotate_unit(float* a, float* b, int u, const KvAppendArgs& g, int64_t pos) {
  if (32 * u >= g.rot) return;
  const float* c = g.cos + pos * (g.rot / 2) + 16 * u;
  const float* s = g.sin + pos * (g.rot / 2) + 16 * u;
  float cc[16], ss[16];
  load_row<DT_F32, 16>(c, 0, cc);
  load_row<DT_F32, 16>(s, 0, ss);
  if (g.inter) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float* p = i < 8 ? a + 2 * i : b + 2 * i - 16;
      const float x = p[0], y = p[1];
      p[0] = __builtin_fmaf(x, cc[i], -(y * ss[i]));
      p[1] = __builtin_fmaf(x, ss[i], y * cc[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float x = a[i], y = b[i];
      a[i] = __builtin_fmaf(x, cc[i], -(y * ss[i]));
      b[i] = __builtin_fmaf(x, ss[i], y * cc[i]);
    }
  }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }

__device__ __forceinline__ uint32_t code(float r, float inv) {
  const float c = fminf(fmaxf(__builtin_rintf(r * inv), -127.0f), 127.0f);
  return (uint32_t)(int)(c + 128.0f);
}

// four codes follow a grown scale (ratio = s_old / s)
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  uint32_t o = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) o |= code((float)((w >> (8 * i)) & 255u) - 128.0f, ratio) << (8 * i);
  return o;
}

// max over the workgroup, in every thread
__device__ __forceinline__ float block_max(float x, float* lds) {
#pragma unroll
  for (int i = 32; i; i >>= 1) x = fmaxf(x, __shfl_xor(x, i));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  float m = lds[0];
#pragma unroll
  for (int i = 1; i < APPEND_THREADS / 64; ++i) m = fmaxf(m, lds[i]);
  return m;
}

// the block's new scale, its inverse, and what its older codes are multiplied by
__device__ __forceinline__ void new_scale(float top, float old, float* s, float* inv, float* ratio) {
  float n = fmaxf(old, top * (1.0f / 127.0f));
  if (n < MIN_SCALE) n = 0.0f;
  *s = n;
  *inv = n > 0.0f ? 1.0f / n : 0.0f;
  *ratio = old * *inv;
}

template <int DT>
__device__ void append_keys(const KvAppendArgs& g, int64_t row0, int64_t pos0, int p0, int n, int64_t id, int h,
                            float* lds, int* bad) {
  const int D = g.c.D, U = D / 32;
  uint8_t* block = g.c.k + (id * g.c.heads + h) * (int64_t)g.c.page * D;
  float* sp = g.c.ks + id * g.c.heads + h;
  const float old = p0 ? *sp : 0.0f;
  float a[16], b[16], top = 0.0f;
  auto fetch = [&](int i) {                                  // unit i of the new rows, rotated; non-finite values are 0
    const int t = i / U, u = i - t * U;
    int d0, d1;
    unit_places(u, g.rot, g.inter, &d0, &d1);
    const int64_t at = (row0 + t) * g.k.ts + h * g.k.hs;
    load_row<DT, 16>(g.k.p, at + d0, a);
    load_row<DT, 16>(g.k.p, at + d1, b);
    rotate_unit(a, b, u, g, pos0 + t);
    int count = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if (!finite(a[e])) a[e] = 0.0f, ++count;
      if (!finite(b[e])) b[e] = 0.0f, ++count;
    }
    return count;
  };
  for (int i = threadIdx.x; i < n * U; i += APPEND_THREADS) {
    *bad += fetch(i);
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, fmaxf(fabsf(a[e]), fabsf(b[e])));
  }
  float s, inv, ratio;
  new_scale(block_max(top, lds), old, &s, &inv, &ratio);
  for (int i = threadIdx.x; i < n * U; i += APPEND_THREADS) {
    fetch(i);
    const int t = i / U, u = i - t * U;
    int d0, d1;
    unit_places(u, g.rot, g.inter, &d0, &d1);
    u32x4 x, y;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      x[w] = y[w] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[w] |= code(a[4 * w + e], inv) << (8 * e);
        y[w] |= code(b[4 * w + e], inv) << (8 * e);
      }
    }
    *(u32x4*)(block + k_byte(p0 + t, d0, D)) = x;
    *(u32x4*)(block + k_byte(p0 + t, d1, D)) = y;
  }
  if (p0 && s != old) {
    for (int i = threadIdx.x; i < p0 * (D / 16); i += APPEND_THREADS) {
      u32x4* p = (u32x4*)(block + k_byte(i / (D / 16), i % (D / 16) * 16, D));
      u32x4 w = *p;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = rescale4(w[e], ratio);
      *p = w;
    }
  }
  if (threadIdx.x == 0) *sp = s;
}

template <int DT>
__device__ void append_values(const KvAppendArgs& g, int64_t row0, int p0, int n, int64_t id, int h, float* lds,
                              int* bad) {
  const int D = g.c.D, F = D / 4;
  uint8_t* block = g.c.v + (id * g.c.heads + h) * (int64_t)g.c.page * D;
  float* sp = g.c.vs + id * g.c.heads + h;
  const float old = p0 ? *sp : 0.0f;
  float top = 0.0f;
  for (int i = threadIdx.x; i < n * F; i += APPEND_THREADS) {
    const int t = i / F, f = i - t * F;
    float r[4];
    load_row<DT, 4>(g.v.p, (row0 + t) * g.v.ts + h * g.v.hs + 4 * f, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (finite(r[e])) top = fmaxf(top, fabsf(r[e]));
      else ++*bad;
    }
  }
  float s, inv, ratio;
  new_scale(block_max(top, lds), old, &s, &inv, &ratio);
  // quads of tokens that hold new ones (and, after a growth, all older ones)
  const int q0 = s != old ? 0 : p0 >> 2, q1 = (p0 + n + 3) >> 2;
  for (int i = threadIdx.x; i < (q1 - q0) * F; i += APPEND_THREADS) {
    const int qd = q0 + i / F, f = i % F;
    u32x4* p = (u32x4*)(block + v_byte(4 * qd, 4 * f, D));
    u32x4 w = {0u, 0u, 0u, 0u};
    if (4 * qd < p0 || 4 * qd + 4 > p0 + n) {
      w = *p;                                                // four tokens a word: older and later ones stay
      if (s != old && 4 * qd < p0) {
        const int keep = min(4, p0 - 4 * qd);                // tokens that follow the scale
        const uint32_t mask = keep == 4 ? 0xFFFFFFFFu : (1u << (8 * keep)) - 1u;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = (rescale4(w[e], ratio) & mask) | (w[e] & ~mask);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = 4 * qd + j - p0;
      if (t >= 0 && t < n) {
        float r[4];
        load_row<DT, 4>(g.v.p, (row0 + t) * g.v.ts + h * g.v.hs + 4 * f, r);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = (w[e] & ~(255u << (8 * j))) | code(finite(r[e]) ? r[e] : 0.0f, inv) << (8 * j);
      }
    }
    *p = w;
  }
  if (threadIdx.x == 0) *sp = s;
}

// Rotate the queries of n tokens (q heads first .. last - 1).
template <int DT>
__device__ void rotate_queries(const KvAppendArgs& g, int64_t row0, int64_t pos0, int n, int first, int last) {
  const int U = g.c.D / 32, per = (last - first) * U;
  for (int i = threadIdx.x; i < n * per; i += APPEND_THREADS) {
    const int t = i / per, j = i - t * per, h = first + j / U, u = j % U;
    int d0, d1;
    unit_places(u, g.rot, g.inter, &d0, &d1);
    float a[16], b[16];
    const int64_t at = (row0 + t) * g.q.ts + h * g.q.hs, to = (row0 + t) * g.qo.ts + h * g.qo.hs;
    load_row<DT, 16>(g.q.p, at + d0, a);
    load_row<DT, 16>(g.q.p, at + d1, b);
    rotate_unit(a, b, u, g, pos0 + t);
    store_row<DT, 16>(g.qo.p, to + d0, a);
    store_row<DT, 16>(g.qo.p, to + d1, b);
  }
}

// grid: x = pages that a sequence's new tokens may touch, y = key heads,
// value heads, then groups of query heads, z = sequences
template <int DT>
__global__ __launch_bounds__(APPEND_THREADS) void append_kernel(KvAppendArgs g, int q_group) {
  __shared__ float lds[APPEND_THREADS / 64];
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
    rotate_queries<DT>(g, row0, first, rotated, h0, min(g.q_heads, h0 + q_group));
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
  if (role < H) append_keys<DT>(g, row0, first, p0, rotated, id, role, lds, &bad);
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
__global__ __launch_bounds__(APPEND_THREADS) void read_kernel(KvReadArgs g) {
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
    const int C = D / 16;
    for (int i = threadIdx.x; i < n * C; i += APPEND_THREADS) {
      const int t = i / C, d = i % C * 16;
      const u32x4 w = *(const u32x4*)(block + k_byte(p0 + t, d, D));
      float r[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) r[e] = value_of(s, (w[e >> 2] >> (8 * (e & 3))) & 255u);
      store_row<DT, 16>(g.k.p, (row0 + t) * g.k.ts + h * g.k.hs + d, r);
    }
  } else {
    const int F = D / 4, q0 = p0 >> 2, q1 = (p0 + n + 3) >> 2;
    for (int i = threadIdx.x; i < (q1 - q0) * F; i += APPEND_THREADS) {
      const int qd = q0 + i / F, d = i % F * 4;
      const u32x4 w = *(const u32x4*)(block + v_byte(4 * qd, d, D));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 4 * qd + j - p0;
        if (t < 0 || t >= n) continue;
        float r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = value_of(s, (w[e] >> (8 * j)) & 255u);
        store_row<DT, 4>(g.v.p, (row0 + t) * g.v.ts + h * g.v.hs + d, r);
      }
    }
  }
}

// pages that `tokens` consecutive tokens can touch, wherever they start
int page_slots(int tokens, int page) { return (int)(((int64_t)tokens + page - 2) / page + 1); }

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& g, hipStream_t st) {
  const int q_group = 8;
  const dim3 grid(page_slots(g.t.max_tokens, g.c.page), 2 * g.c.heads + (g.q.p ? (g.q_heads + q_group - 1) / q_group : 0),
                  g.t.batch);
  if (g.dtype == DT_F16) append_kernel<DT_F16><<<grid, APPEND_THREADS, 0, st>>>(g, q_group);
  else if (g.dtype == DT_BF16) append_kernel<DT_BF16><<<grid, APPEND_THREADS, 0, st>>>(g, q_group);
  else append_kernel<DT_F32><<<grid, APPEND_THREADS, 0, st>>>(g, q_group);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvReadArgs& g, hipStream_t st) {
  const dim3 grid(page_slots(g.t.max_tokens, g.c.page), 2 * g.c.heads, g.t.batch);
  if (g.dtype == DT_F16) read_kernel<DT_F16><<<grid, APPEND_THREADS, 0, st>>>(g);
  else if (g.dtype == DT_BF16) read_kernel<DT_BF16><<<grid, APPEND_THREADS, 0, st>>>(g);
  else read_kernel<DT_F32><<<grid, APPEND_THREADS, 0, st>>>(g);
  return hipGetLastError();
}

}  // namespace lowbit
