// gfx950 products of a few rows (M <= 16) with 4-bit group-scaled weights:
// Y = act(X W^T + bias), W = s (q - z) with an FP16 scale and zero point per
// 128 weights along K (the text encoder's format, "Como Bonsai Ternary 4B
// revoluciona la difusion texto-imagen", section "Arquitectura de despliegue
// y eficiencia en tiempo de ejecucion"). It is the form for single tokens:
// one launch, no workspace, bound by reading the codes once.
//
// Mathematics. A code enters v_mfma_f32_16x16x32 as 16 + q, which is exact in
// both 16-bit types with q in the top four mantissa bits (FP16 0x4C00 | q << 6,
// BF16 0x4180 | q << 3): one shift and one AND-OR for two weights. With
// P = sum x (16 + q) and sx = sum x over a group (an MFMA against ones),
//   sum x s (q - z) = s (P - (16 + z) sx),
// in FP32. The offset of 16 (and not the 128 of the lowest mantissa bits)
// keeps the cancellation within about four times the size of the terms.
#include "common.h"

namespace lowbit {

namespace gemv {
constexpr int MAXWAVES = 16;
}

template <bool BF16>
__device__ __forceinline__ u32x4 gemv_codes(uint32_t w) {
  constexpr uint32_t mask = BF16 ? 0x00780078u : 0x03C003C0u, base = BF16 ? 0x41804180u : 0x4C004C00u;
  u32x4 r;
  if constexpr (BF16) {
    r[0] = ((w << 3) & mask) | base;
    r[1] = ((w >> 1) & mask) | base;
    r[2] = ((w >> 5) & mask) | base;
    r[3] = ((w >> 9) & mask) | base;
  } else {
    r[0] = ((w << 6) & mask) | base;
    r[1] = ((w << 2) & mask) | base;
    r[2] = ((w >> 2) & mask) | base;
    r[3] = ((w >> 6) & mask) | base;
  }
  return r;
}

// A workgroup of `blockDim.x / 64` waves owns batches of T tiles of 16
// columns; wave w holds the activations of GPW groups of K as MFMA operands
// in registers (the whole of X once per workgroup, over all its batches,
// while K is at most waves * GPW groups; longer K goes chunk by chunk).
// Codes: lane (q, c) loads 16 bytes, a quarter of column c's group, so a
// wave-wide load reads 64 contiguous bytes of 16 columns; a 4 x 4 exchange
// between the lane groups then gives step s the words 4 s + q, so that the
// activations' loads cover 64 contiguous bytes of each row too. All code
// loads of a batch are issued before the first is used. The waves' partial
// tiles are added in LDS in wave order (deterministic).
template <bool BF16, int GPW, int T>
__global__ __launch_bounds__(64 * gemv::MAXWAVES) void gemv_int4_kernel(GemmArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  f32x4* red = (f32x4*)smem;                                // [waves][T][64]
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int q = lane >> 4, c16 = lane & 15;
  const int G = a.K >> 7;
  const int tiles = (a.N + 15) >> 4, batches = (tiles + T - 1) / T;
  const int per = waves * GPW;                              // groups in one chunk
  const uint16_t* xrow = a.X + (int64_t)min(c16, a.M - 1) * a.ldx + 8 * q;
  constexpr uint32_t one = BF16 ? 0x3F803F80u : 0x3C003C00u;
  const u32x4 ones = {one, one, one, one};
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  u32x4 xf[GPW][4];
  f32x4 sx[GPW];
  for (int batch = blockIdx.x; batch < batches; batch += gridDim.x) {
    f32x4 acc[T];
#pragma unroll
    for (int t = 0; t < T; ++t) acc[t] = zero;
    for (int g0 = 0; g0 < G; g0 += per) {
      const int gw = g0 + wave * GPW;                       // first group of this wave
      const int ng = min(GPW, G - gw);                      // may be <= 0: nothing to add
      if (ng > 0) {
        u32x4 cw[T][GPW];
        uint32_t sr[T], zr[T];
#pragma unroll
        for (int t = 0; t < T; ++t) {
          const int64_t n = min((batch * T + t) * 16 + c16, a.N - 1);
          const uint8_t* wp = a.W + n * (a.K >> 1) + 16 * q;
#pragma unroll
          for (int u = 0; u < GPW; ++u) cw[t][u] = *(const u32x4*)(wp + (gw + min(u, ng - 1)) * 64);
          const int64_t at = n * G + gw + min(q, ng - 1);
          sr[t] = a.S[at];
          zr[t] = a.Z[at];
        }
        if (batch == (int)blockIdx.x || per < G) {
#pragma unroll
          for (int u = 0; u < GPW; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) xf[u][s] = *(const u32x4*)(xrow + (gw + min(u, ng - 1)) * 128 + 32 * s);
#pragma unroll
          for (int u = 0; u < GPW; ++u) {
            sx[u] = zero;
#pragma unroll
            for (int s = 0; s < 4; ++s) sx[u] = mfma16<BF16>(xf[u][s], ones, sx[u]);
          }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
#pragma unroll
          for (int u = 0; u < GPW; ++u) {
            auto x = __builtin_amdgcn_permlane32_swap(cw[t][u][0], cw[t][u][2], false, false);
            auto y = __builtin_amdgcn_permlane32_swap(cw[t][u][1], cw[t][u][3], false, false);
            auto e = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
            auto o = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
            const uint32_t w[4] = {e[0], e[1], o[0], o[1]};
            f32x4 p = zero;
#pragma unroll
            for (int s = 0; s < 4; ++s) p = mfma16<BF16>(xf[u][s], gemv_codes<BF16>(w[s]), p);
            // the scale and zero point of group gw + u sit in lane group u
            const float s_ = half_bits_to_float((uint16_t)__shfl((int)sr[t], 16 * u + c16));
            const float z_ = half_bits_to_float((uint16_t)__shfl((int)zr[t], 16 * u + c16));
            if (u < ng) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[t][i] = __builtin_fmaf(s_, __builtin_fmaf(-(16.0f + z_), sx[u][i], p[i]), acc[t][i]);
            }
          }
        }
      }
    }
    if (waves > 1) {
#pragma unroll
      for (int t = 0; t < T; ++t) red[(wave * T + t) * 64 + lane] = acc[t];
      __syncthreads();
    }
    // tile t of the batch is finished by wave t (mod waves); a lane holds rows 4q + i of column n
    for (int t = wave; t < T; t += waves) {
      f32x4 sum;
      if (waves > 1) {
        sum = red[t * 64 + lane];
        for (int w = 1; w < waves; ++w) sum += red[(w * T + t) * 64 + lane];
      } else {
        sum = acc[0];
#pragma unroll
        for (int k = 1; k < T; ++k)
          if (t == k) sum = acc[k];
      }
      const int n = (batch * T + t) * 16 + c16;
      if (n < a.N) {
        const float b = a.bias ? load_bias(a.bias, a.bias_dtype, n) : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * q + i < a.M) store_out(a.Y, a.ldy, a.y_dtype, 4 * q + i, n, finish(sum[i], b, a.act));
      }
    }
    if (waves > 1 && batch + (int)gridDim.x < batches) __syncthreads();
  }
}

namespace {

template <bool BF16, int GPW, int T>
void run(const GemmArgs& a, int waves, int blocks, hipStream_t st) {
  gemv_int4_kernel<BF16, GPW, T><<<dim3(blocks), dim3(64 * waves), (size_t)waves * T * 1024, st>>>(a);
}

template <bool BF16>
void dispatch(const GemmArgs& a, int num_cu, hipStream_t st) {
  const int G = a.K / 128, tiles = (a.N + 15) / 16;
  const int waves = min(gemv::MAXWAVES, (G + 1) / 2);
  const int t = tiles <= 2 * num_cu ? 1 : 2;
  const int blocks = min((tiles + t - 1) / t, 2 * num_cu);
  if (t == 1) run<BF16, 2, 1>(a, waves, blocks, st);
  else run<BF16, 2, 2>(a, waves, blocks, st);
}

}  // namespace

hipError_t launch_gemv_int4(bool x_bf16, const GemmArgs& a, int num_cu, hipStream_t st) {
  if (x_bf16) dispatch<true>(a, num_cu, st);
  else dispatch<false>(a, num_cu, st);
  return hipGetLastError();
}

}  // namespace lowbit
