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
constexpr int MAXWAVES = 12;               // of a workgroup
constexpr int CU_WAVES = 16;               // waves that a CU holds at the registers of GPW = 3 (124)
constexpr int RING = 2;                    // tiles in flight a wave (3 to 5 are no faster)
constexpr int BATCH = 16;                  // tiles between two visits of a chunk of K
constexpr int slot_bytes(int gpw) { return gpw * 1024 + 512; }   // codes, then scales and zero points (4-byte slots)
// LDS: rings of the waves, partial tiles [2][waves], biases [2][BATCH][16], running tiles [BATCH] for several chunks
constexpr size_t lds_bytes(int gpw, int waves, int chunks) {
  return (size_t)waves * RING * slot_bytes(gpw) + (size_t)2 * waves * 1024 + 2 * BATCH * 64 + (chunks > 1 ? BATCH * 1024 : 0);
}
}  // namespace gemv

template <int N>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

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

// A workgroup's waves split K: wave w holds the activations of GPW groups as
// MFMA operands in registers, and the workgroup walks its tiles of 16 columns
// (blockIdx.x, + gridDim.x, ...), the waves' partial tiles added in LDS in
// wave order (deterministic). K beyond waves * GPW groups goes chunk by chunk
// over batches of tiles, so that activations are read once per batch.
//
// Bound by the memory pipeline of a CU, so few and wide requests:
//  * Codes go global -> LDS by DMA into a ring of the wave's own (no barrier
//    and no registers), RING tiles deep: lane (q, c) fetches a quarter of
//    column c's group, 64 contiguous bytes of 16 columns an instruction. MFMA
//    step s then reads word q of quarter s (64 consecutive words), so that
//    the activations' loads cover 64 contiguous bytes of each row too.
//  * Scales and zero points: one DMA each for four groups of 16 columns. As
//    register loads per group they took as long as the codes: 131072 x 2560
//    at M = 2 took 54 us, 44 without them.
template <bool BF16, int GPW>
__global__ __launch_bounds__(64 * gemv::MAXWAVES) void gemv_int4_kernel(GemmArgs a, int chunks) {
  constexpr int SLOT = gemv::slot_bytes(GPW), RING = gemv::RING, BATCH = gemv::BATCH, LOADS = GPW + 2;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int q = lane >> 4, c16 = lane & 15;
  uint8_t* ring = smem + wave * RING * SLOT;
  f32x4* red = (f32x4*)(smem + waves * RING * SLOT);        // [2][waves][64]
  float* bias = (float*)(red + 2 * waves * 64);             // [2][BATCH][16]
  f32x4* run = (f32x4*)(bias + 2 * BATCH * 16);             // [BATCH][64]
  const int G = a.K >> 7;
  const int tiles = (a.N + 15) >> 4, nb = gridDim.x;
  const int te = (tiles - 1 - (int)blockIdx.x) / nb + 1;    // tiles of this workgroup
  const int items = te * chunks;
  const uint16_t* xrow = a.X + (int64_t)min(c16, a.M - 1) * a.ldx + 8 * q;
  constexpr uint32_t one = BF16 ? 0x3F803F80u : 0x3C003C00u;
  const u32x4 ones = {one, one, one, one};
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

  // order of the work: batch of tiles, chunk of K, tile
  struct Item { int tile, chunk, first; };
  auto advance = [&](Item& i) __attribute__((always_inline)) {
    if (++i.tile == min(i.first + BATCH, te)) {
      if (++i.chunk == chunks) {
        i.chunk = 0;
        i.first = i.tile;
      } else {
        i.tile = i.first;
      }
    }
  };
  // first group of this wave in a chunk; groups past the end repeat the last one (and count for nothing)
  auto group0 = [&](int chunk) __attribute__((always_inline)) { return (chunk * waves + wave) * GPW; };
  auto fetch = [&](const Item& i, int slot) __attribute__((always_inline)) {
    const uint32_t n = min((blockIdx.x + i.tile * nb) * 16 + c16, (uint32_t)a.N - 1);
    const int gw = group0(i.chunk);
    const uint32_t wo = n * ((uint32_t)a.K >> 1) + 16 * q;  // codes span less than 4 GiB
    const uint32_t so = (n * (uint32_t)G + (uint32_t)min(gw + min(q, GPW - 1), G - 1)) * 2;
    const uint32_t to = lds_addr(ring + slot * SLOT);
#pragma unroll
    for (int u = 0; u < GPW; ++u) dma_lds16(a.W, wo + (uint32_t)min(gw + u, G - 1) * 64, to + u * 1024);
    dma_lds2(a.S, so, to + GPW * 1024);
    dma_lds2(a.Z, so, to + GPW * 1024 + 256);
  };

  u32x4 xf[GPW][4];
  f32x4 sx[GPW];
  Item in{0, 0, 0}, at{0, 0, 0};                            // next to fetch, next to compute
#pragma unroll
  for (int r = 0; r < RING; ++r)
    if (r < items) {
      fetch(in, r);
      advance(in);
    }
  int slot = 0, buf = 0;
  for (int i = 0; i < items; ++i) {
    const int gw = group0(at.chunk), tb = at.tile - at.first;
    if (tb == 0) {                                          // wave-uniform: a new batch or chunk
      if (at.chunk == 0 && a.bias) {
        for (int k = tid; k < BATCH * 16; k += blockDim.x) {
          const int nk = (blockIdx.x + (at.first + (k >> 4)) * nb) * 16 + (k & 15);
          bias[((at.first / BATCH) & 1) * BATCH * 16 + k] =
              (at.first + (k >> 4) < te && nk < a.N) ? load_bias(a.bias, a.bias_dtype, nk) : 0.0f;
        }
      }
      if (i == 0 || chunks > 1) {
#pragma unroll
        for (int u = 0; u < GPW; ++u)
#pragma unroll
          for (int s = 0; s < 4; ++s) xf[u][s] = *(const u32x4*)(xrow + (int64_t)min(gw + u, G - 1) * 128 + 32 * s);
#pragma unroll
        for (int u = 0; u < GPW; ++u) {
          sx[u] = zero;
#pragma unroll
          for (int s = 0; s < 4; ++s) sx[u] = mfma16<BF16>(xf[u][s], ones, sx[u]);
        }
      }
    }
    // this item's loads are done; those of the next RING - 1 items may be in flight
    if (items - i >= RING) wait_loads<(RING - 1) * LOADS>();
    else wait_loads<0>();
    const uint8_t* from = ring + slot * SLOT;
    f32x4 acc = zero;
#pragma unroll
    for (int u = 0; u < GPW; ++u) {
      f32x4 p = zero;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        p = mfma16<BF16>(xf[u][s], gemv_codes<BF16>(*(const uint32_t*)(from + u * 1024 + (s * 16 + c16) * 16 + q * 4)), p);
      const float sc = half_bits_to_float(*(const uint16_t*)(from + GPW * 1024 + (u * 16 + c16) * 4));
      const float ze = half_bits_to_float(*(const uint16_t*)(from + GPW * 1024 + 256 + (u * 16 + c16) * 4));
      const float s_ = gw + u < G ? sc : 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(s_, __builtin_fmaf(-(16.0f + ze), sx[u][e], p[e]), acc[e]);
    }
    if (i + RING < items) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");    // the slot has been read
      fetch(in, slot);
      advance(in);
    }
    slot = slot + 1 == RING ? 0 : slot + 1;
    if (waves > 1) {
      red[(buf * waves + wave) * 64 + lane] = acc;
      __syncthreads();
    }
    // tile tb of a batch is finished by wave tb (mod waves), in every chunk. The other buffer of partials takes
    // the next item meanwhile: its last readers have passed the barrier above.
    if (tb % waves == wave) {
      if (waves > 1) {
        acc = red[buf * waves * 64 + lane];
        for (int w = 1; w < waves; ++w) acc += red[(buf * waves + w) * 64 + lane];
      }
      if (at.chunk) acc += run[tb * 64 + lane];
      if (at.chunk + 1 < chunks) {
        run[tb * 64 + lane] = acc;
      } else {
        const int n = (blockIdx.x + at.tile * nb) * 16 + c16;   // a lane holds rows 4q + e of column n
        if (n < a.N) {
          const float b = a.bias ? bias[(((at.first / BATCH) & 1) * BATCH + tb) * 16 + c16] : 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (4 * q + e < a.M) store_out(a.Y, a.ldy, a.y_dtype, 4 * q + e, n, finish(acc[e], b, a.act));
        }
      }
    }
    buf ^= 1;
    advance(at);
  }
}

namespace {

template <bool BF16, int GPW>
void run(const GemmArgs& a, int num_cu, hipStream_t st) {
  const int G = a.K / 128, tiles = (a.N + 15) / 16;
  const int chunks = (G + GPW * gemv::MAXWAVES - 1) / (GPW * gemv::MAXWAVES);
  const int waves = (G + GPW * chunks - 1) / (GPW * chunks);
  const size_t lds = gemv::lds_bytes(GPW, waves, chunks);
  const int per_cu = max(1, min(gemv::CU_WAVES / waves, (int)(160 * 1024 / lds)));
  gemv_int4_kernel<BF16, GPW><<<dim3(min(tiles, per_cu * num_cu)), dim3(64 * waves), lds, st>>>(a, chunks);
}

// Groups a wave: more waves hide more latency, fewer leave less to add. At
// 131072 x 2560 (20 groups), M = 2, 1 / 2 / 3 / 4 groups a wave took 64 / 45 /
// 41 / 54 us (three: two workgroups a CU). With few tiles a CU one workgroup of
// two groups a wave balances better and reads the activations once: 19456 x
// 2560, M = 16, 14.9 / 12.5 / 14.2 / 16.9. Short K takes fewer so that a
// workgroup has waves at all.
template <bool BF16>
void dispatch(const GemmArgs& a, int num_cu, hipStream_t st) {
  const int G = a.K / 128, tiles = (a.N + 15) / 16;
  if (G <= 4) run<BF16, 1>(a, num_cu, st);
  else if (G <= 12 || (G <= 2 * gemv::MAXWAVES && tiles <= 8 * num_cu)) run<BF16, 2>(a, num_cu, st);
  else run<BF16, 3>(a, num_cu, st);
}

}  // namespace

hipError_t launch_gemv_int4(bool x_bf16, const GemmArgs& a, int num_cu, hipStream_t st) {
  if (x_bf16) dispatch<true>(a, num_cu, st);
  else dispatch<false>(a, num_cu, st);
  return hipGetLastError();
}

}  // namespace lowbit
