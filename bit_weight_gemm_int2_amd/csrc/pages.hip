// The pages of the paged cache: new tables of pages for the sequences that go on
// (forking, dropping and trimming them, making room, moving pages to the front
// of the pool) and copying pages as such a table asks for.
//
// A new table is a function of the old one, the lengths and the rows that go on,
// worked out on the device: no counters live from call to call, and a page is
// free when no slot of the new sequences refers to it. The steps:
//   clear   the sets of pages; the owners of the last, partly filled pages
//   mark    every kept slot's page as used; as whole where it is no partly
//           filled last page; the lowest row of a partly filled page as its owner
//   scan    used pages before each word of 32; the slots that need a new page
//           before each row; the lowest free pages, as many as are needed
//   apply   table, lengths, pairs to copy, counts
// A last, partly filled page is the row's own when no whole reference to it is
// left and no lower row has it too; else the row copies it (the next tokens go
// there). The sets are bitmaps: their updates (or, min) do not depend on the order.
#include <algorithm>

#include "pages.h"

namespace lowbit {

namespace {

constexpr int SCAN_THREADS = 1024;

__device__ __forceinline__ uint32_t get(const uint32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ int32_t get(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ void put(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// One new row: the old row that it continues, its tokens, and the slots
// [grow0, grow1) that its room takes beyond them.
struct Row {
  int64_t at;               // of the old row in the old table
  int len, part;            // part: the slot of a partly filled last page, -1 where there is none
  int grow0, grow1;
};

__device__ __forceinline__ Row find_row(const RemapArgs& g, int c) {
  const int r = g.rows ? g.rows[c] : c;
  Row w;
  const bool goes = r >= 0 && r < g.batch;
  w.at = goes ? (int64_t)r * g.width : 0;
  w.len = goes ? max(0, min(g.lens[r], g.most)) : 0;
  const int whole = w.len >> g.shift, rest = w.len & (g.page - 1);
  w.part = rest ? whole : -1;
  w.grow0 = whole + (rest != 0);
  const int64_t end = (int64_t)w.len + (g.room ? max(0, g.room[c]) : 0);
  w.grow1 = max(w.grow0, (int)min(g.width_out, (end + g.page - 1) >> g.shift));
  return w;
}

// The page that slot s of row w keeps, or -1.
__device__ __forceinline__ int kept(const RemapArgs& g, const Row& w, int s) {
  const int64_t first = (int64_t)s << g.shift;
  if (first >= w.len) return -1;
  const int id = g.table[w.at + s];
  if (id < 0 || id >= g.pages) return -1;
  // no token of it is among the first `sinks`, nor is one seen from position len on
  if (g.window && s != w.part && first >= g.sinks && first + g.page - 1 <= w.len - g.window) return -1;
  return id;
}

__device__ __forceinline__ bool copies(const RemapArgs& g, int c, int id) {
  return id >= 0 && ((get(g.whole + (id >> 5)) >> (id & 31) & 1) || get(g.owner + id) != c);
}

__device__ void clear(const RemapArgs& g, int64_t tid, int64_t threads) {
  for (int64_t i = tid; i < g.words; i += threads) {
    put(g.used + i, 0u);
    put(g.whole + i, 0u);
  }
  for (int64_t c = tid; c < g.new_batch; c += threads) {
    const Row w = find_row(g, (int)c);
    const int id = w.part >= 0 ? kept(g, w, w.part) : -1;
    if (id >= 0) put(g.owner + id, 0x7fffffff);
  }
}

__device__ void mark(const RemapArgs& g, int64_t tid, int64_t threads) {
  const int slots = (int)min(g.width, g.width_out);
  for (int64_t i = tid; i < (int64_t)g.new_batch * slots; i += threads) {
    const int c = (int)((uint32_t)i / (uint32_t)slots), s = (int)((uint32_t)i % (uint32_t)slots);
    const Row w = find_row(g, c);
    const int id = kept(g, w, s);
    if (id < 0) continue;
    const uint32_t bit = 1u << (id & 31);
    __hip_atomic_fetch_or(g.used + (id >> 5), bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (s != w.part) __hip_atomic_fetch_or(g.whole + (id >> 5), bit, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    else __hip_atomic_fetch_min(g.owner + id, c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// What a thread's value adds to before it, and the workgroup's total.
__device__ __forceinline__ int2 scan2(int2 v, int2* lds, int2* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int2 x = v;
#pragma unroll
  for (int i = 1; i < 64; i <<= 1) {
    const int a = __shfl_up(x.x, i), b = __shfl_up(x.y, i);
    if (lane >= i) x.x += a, x.y += b;
  }
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int2 before = {0, 0}, all = {0, 0};
  for (int k = 0; k < SCAN_THREADS / 64; ++k) {
    const int2 y = lds[k];
    if (k < wave) before.x += y.x, before.y += y.y;
    all.x += y.x, all.y += y.y;
  }
  __syncthreads();
  *total = all;
  return {before.x + x.x - v.x, before.y + x.y - v.y};
}

__device__ __forceinline__ int rank_of(const RemapArgs& g, int p) {   // used pages below p
  if (p >= g.pages) return g.info->used;
  return g.before[p >> 5] + __popc(get(g.used + (p >> 5)) & ((1u << (p & 31)) - 1u));
}

// One workgroup of SCAN_THREADS.
__device__ void scan(const RemapArgs& g) {
  __shared__ int2 lds[SCAN_THREADS / 64];
  __shared__ int done;
  const int tid = threadIdx.x;
  int2 total, run = {0, 0};
  for (int64_t b = 0; b < g.words; b += SCAN_THREADS) {
    const int64_t i = b + tid;
    const int2 mine = {i < g.words ? __popc(get(g.used + i)) : 0, 0};
    const int2 at = scan2(mine, lds, &total);
    if (i < g.words) g.before[i] = run.x + at.x;
    run.x += total.x;
  }
  const int used = run.x;
  run = {0, 0};
  for (int64_t b = 0; b < g.new_batch; b += SCAN_THREADS) {
    const int64_t c = b + tid;
    int2 mine = {0, 0};
    if (c < g.new_batch) {
      const Row w = find_row(g, (int)c);
      mine.y = w.part >= 0 && copies(g, (int)c, kept(g, w, w.part));
      mine.x = mine.y + w.grow1 - w.grow0;
    }
    const int2 at = scan2(mine, lds, &total);
    if (c < g.new_batch) {
      g.need[c] = run.x + at.x;
      g.copy[c] = mine.y ? run.y + at.y : -1;
    }
    run.x += total.x;
    run.y += total.y;
  }
  const int need = run.x, fresh = min(need, (int)g.pages - used), n = used + fresh;
  if (tid == 0) {
    g.info->used = used;
    done = 0;
  }
  __syncthreads();
  const int moves = g.compact ? used - rank_of(g, n) : 0;
  // copies of rows whose turn comes before the free pages run out
  int mine = 0;
  for (int64_t c = tid; c < g.new_batch; c += SCAN_THREADS) mine += g.copy[c] >= 0 && g.need[c] < fresh;
  if (mine) atomicAdd(&done, mine);
  // the lowest free pages: the first `moves` of them take the pages that move
  const int take = moves + fresh;
  for (int64_t i = tid; i < g.words; i += SCAN_THREADS) {
    int at = (int)(32 * i) - g.before[i];
    if (at >= take) break;                                   // free pages before a word never get fewer
    uint32_t free = ~get(g.used + i);
    for (; free && at < take; free &= free - 1, ++at) {
      const int64_t p = 32 * i + __ffs(free) - 1;
      if (p < g.pages) g.free[at] = (int)p;
    }
  }
  __syncthreads();
  if (tid == 0) {
    g.info->fresh = fresh;
    g.info->n = n;
    g.info->moves = moves;
    g.info->pairs = moves + done;
    g.counts[0] = moves + done;
    g.counts[1] = n;
    g.counts[2] = need - fresh;
    g.counts[3] = moves;
  }
}

__device__ void apply(const RemapArgs& g, int64_t tid, int64_t threads) {
  const int fresh = g.info->fresh, n = g.info->n, moves = g.info->moves, pairs = g.info->pairs;
  const int below = g.info->used - moves;                    // used pages that stay below n
  const int wide = (int)g.width_out;
  for (int64_t i = tid; i < (int64_t)g.new_batch * wide; i += threads) {
    const int c = (int)((uint32_t)i / (uint32_t)wide), s = (int)((uint32_t)i % (uint32_t)wide);
    const Row w = find_row(g, c);
    int id = kept(g, w, s), nth = -1;
    const bool copy = s == w.part && g.copy[c] >= 0;
    if (copy) nth = g.need[c];
    else if (s >= w.grow0 && s < w.grow1) nth = g.need[c] + (g.copy[c] >= 0) + s - w.grow0;
    if (nth >= 0) {
      const int to = nth < fresh ? g.free[moves + nth] : -1;
      if (copy && to >= 0) {
        g.src[moves + g.copy[c]] = id;
        g.dst[moves + g.copy[c]] = to;
      }
      id = to;
    } else if (moves && id >= n) {
      id = g.free[rank_of(g, id) - below];
    }
    g.table_out[i] = id;
    if (s == 0) g.lens_out[c] = w.len;
  }
  if (!wide)
    for (int64_t c = tid; c < g.new_batch; c += threads) g.lens_out[c] = 0;
  if (moves) {
    for (int64_t i = (n >> 5) + tid; i < g.words; i += threads) {
      uint32_t bits = get(g.used + i);
      if (i == n >> 5) bits &= ~((1u << (n & 31)) - 1u);
      for (; bits; bits &= bits - 1) {
        const int p = (int)(32 * i) + __ffs(bits) - 1, k = rank_of(g, p) - below;
        g.src[k] = p;
        g.dst[k] = g.free[k];
      }
    }
  }
  for (int64_t i = pairs + tid; i < g.capacity; i += threads) g.src[i] = g.dst[i] = -1;
}

__global__ __launch_bounds__(256) void remap_clear_kernel(RemapArgs g) {
  clear(g, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}
__global__ __launch_bounds__(256) void remap_mark_kernel(RemapArgs g) {
  mark(g, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}
__global__ __launch_bounds__(SCAN_THREADS) void remap_scan_kernel(RemapArgs g) { scan(g); }
__global__ __launch_bounds__(256) void remap_apply_kernel(RemapArgs g) {
  apply(g, (int64_t)blockIdx.x * 256 + threadIdx.x, (int64_t)gridDim.x * 256);
}

// All steps by one workgroup, for small tables.
__global__ __launch_bounds__(SCAN_THREADS) void remap_kernel(RemapArgs g) {
  clear(g, threadIdx.x, SCAN_THREADS);
  __syncthreads();
  mark(g, threadIdx.x, SCAN_THREADS);
  __syncthreads();
  scan(g);
  __syncthreads();
  apply(g, threadIdx.x, SCAN_THREADS);
}

// A pair's blocks (all heads of a page lie together) in pieces of PIECE bytes,
// keys' first, then values'; the pair's first piece brings the scales too.
constexpr int PIECE = 16384;

__global__ __launch_bounds__(256) void copy_pages_kernel(KvCache c, const int32_t* src, const int32_t* dst, int pairs,
                                                         const int32_t* count) {
  const int bytes = c.heads * c.page * c.D;                  // of a page's keys
  const int pieces = (bytes + PIECE - 1) / PIECE;
  const int n = count ? max(0, min(*count, pairs)) : pairs;
  for (int64_t item = blockIdx.x; item < (int64_t)n * 2 * pieces; item += gridDim.x) {
    const int pair = (int)(item / (2 * pieces)), part = (int)(item - (int64_t)pair * 2 * pieces);
    const int64_t from = src[pair], to = dst[pair];
    if (from < 0 || from >= c.pages || to < 0 || to >= c.pages || from == to) continue;
    uint8_t* const base = part < pieces ? c.k : c.v;
    const int at = (part < pieces ? part : part - pieces) * PIECE + threadIdx.x * 16;
    const uint8_t* a = base + from * bytes + at;
    uint8_t* b = base + to * bytes + at;
    u32x4 w[PIECE / 4096];
#pragma unroll
    for (int i = 0; i < PIECE / 4096; ++i)
      if (at + 4096 * i < bytes) w[i] = __builtin_nontemporal_load((const u32x4*)(a + 4096 * i));
#pragma unroll
    for (int i = 0; i < PIECE / 4096; ++i)
      if (at + 4096 * i < bytes) __builtin_nontemporal_store(w[i], (u32x4*)(b + 4096 * i));
    if (part == 0) {
      for (int h = threadIdx.x; h < c.heads; h += 256) {
        c.ks[to * c.heads + h] = c.ks[from * c.heads + h];
        c.vs[to * c.heads + h] = c.vs[from * c.heads + h];
      }
    }
  }
}

size_t up(size_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

size_t remap_workspace(int64_t new_batch, int64_t pages) {
  const size_t words = (pages + 31) / 32;
  return 256 + 3 * up(4 * words) + 2 * up(4 * pages) + 2 * up(4 * new_batch);
}

hipError_t launch_remap(RemapArgs g, void* workspace, int num_cu, hipStream_t st) {
  g.words = (g.pages + 31) / 32;
  uint8_t* p = (uint8_t*)workspace;
  auto take = [&](size_t bytes) {
    uint8_t* q = p;
    p += up(bytes);
    return q;
  };
  g.info = (RemapInfo*)take(256);
  g.used = (uint32_t*)take(4 * g.words);
  g.whole = (uint32_t*)take(4 * g.words);
  g.before = (int32_t*)take(4 * g.words);
  g.owner = (int32_t*)take(4 * g.pages);
  g.free = (int32_t*)take(4 * g.pages);
  g.need = (int32_t*)take(4 * g.new_batch);
  g.copy = (int32_t*)take(4 * g.new_batch);
  const int64_t slots = g.new_batch * std::max(g.width_out, g.width);
  if (slots <= 16384 && g.pages <= 65536) {
    remap_kernel<<<1, SCAN_THREADS, 0, st>>>(g);
    return hipGetLastError();
  }
  auto blocks = [&](int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 8 * num_cu)); };
  remap_clear_kernel<<<blocks(std::max(g.words, (int64_t)g.new_batch)), 256, 0, st>>>(g);
  remap_mark_kernel<<<blocks(slots), 256, 0, st>>>(g);
  remap_scan_kernel<<<1, SCAN_THREADS, 0, st>>>(g);
  remap_apply_kernel<<<blocks(std::max(slots, g.words)), 256, 0, st>>>(g);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const KvCache& c, const int32_t* src, const int32_t* dst, int pairs, const int32_t* count,
                             int num_cu, hipStream_t st) {
  const int64_t pieces = ((int64_t)c.heads * c.page * c.D + PIECE - 1) / PIECE * 2;
  copy_pages_kernel<<<(unsigned)std::min<int64_t>(pairs * pieces, 8 * num_cu), 256, 0, st>>>(c, src, dst, pairs, count);
  return hipGetLastError();
}

}  // namespace lowbit
