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
  int row;                  // the old row, 0 where there is none
  int len, part;            // part: the slot of a partly filled last page, -1 where there is none
  int grow0, grow1;
};

__device__ __forceinline__ Row find_row(const RemapArgs& g, int c) {
  const int r = g.rows ? g.rows[c] : c;
  Row w;
  const bool goes = r >= 0 && r < g.batch;
  w.row = goes ? r : 0;
  w.at = w.row * g.width;
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

// The sum of x over the lanes up to this one, by DPP moves: within rows of 16
// lanes, then the last lane of a row to the next row, and of two rows to the others.
template <int CTRL, int ROWS>
__device__ __forceinline__ int moved(int x) { return __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xf, false); }
__device__ __forceinline__ int row_sums(int x) {
  x += moved<0x111, 0xf>(x);
  x += moved<0x112, 0xf>(x);
  x += moved<0x114, 0xf>(x);
  return x + moved<0x118, 0xf>(x);
}
__device__ __forceinline__ int wave_sums(int x) {
  x = row_sums(x);
  x += moved<0x142, 0xa>(x);
  return x + moved<0x143, 0xc>(x);
}

// What a thread's values add to before it, and the workgroup's totals (of 16 waves).
__device__ __forceinline__ int2 scan2(int2 v, int2* lds, int2* total) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int2 x = {wave_sums(v.x), wave_sums(v.y)};
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  int2 y = lds[lane & 15];                                   // every row of 16 lanes holds the 16 waves' sums
  y = {row_sums(y.x), row_sums(y.y)};
  __syncthreads();
  *total = {__builtin_amdgcn_readlane(y.x, 15), __builtin_amdgcn_readlane(y.y, 15)};
  const int before = max(wave - 1, 0);
  const int2 base = {__builtin_amdgcn_readlane(y.x, before), __builtin_amdgcn_readlane(y.y, before)};
  return {(wave ? base.x : 0) + x.x - v.x, (wave ? base.y : 0) + x.y - v.y};
}
static_assert(SCAN_THREADS == 16 * 64, "one row of lanes holds the waves' sums");

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
  for (int64_t p = tid; p < g.pages; p += SCAN_THREADS) {
    const int at = (int)p - rank_of(g, (int)p);
    if (at >= take) break;                                   // free pages before a page never get fewer
    if (!(get(g.used + (p >> 5)) >> (p & 31) & 1)) g.free[at] = (int)p;
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
    for (int64_t p = n + tid; p < g.pages; p += threads) {
      if (!(get(g.used + (p >> 5)) >> (p & 31) & 1)) continue;
      const int k = rank_of(g, (int)p) - below;
      g.src[k] = (int)p;
      g.dst[k] = g.free[k];
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

// The steps by one workgroup with the sets and the rows in LDS, the last one
// (APPLY) for small tables only. Bound by latency (rows, lengths and table one
// after the other, then the table again for the new one) and, for larger tables,
// by the instructions of one CU: a power of two of lanes, as wide as a row or 64,
// walks the slots of a row, so that there is no division, with BATCH entries in
// flight.
constexpr int BATCH = 4;

// The slots of rows c, c + step, ... that a thread takes: s0, s0 + lanes, ... of
// each. WIDE: 64 lanes a row, whose number and values are the same in all of a wave.
template <bool WIDE>
struct Walk {
  int c, s, wide, step, s0, lanes;
  __device__ __forceinline__ Walk(int slots, int log_lanes) {
    if (WIDE) log_lanes = 6;
    lanes = 1 << log_lanes;
    s0 = threadIdx.x & (lanes - 1);
    s = 0;
    c = threadIdx.x >> log_lanes;
    if (WIDE) c = __builtin_amdgcn_readfirstlane(c);
    step = SCAN_THREADS >> log_lanes;
    wide = slots;
  }
  __device__ __forceinline__ bool any(int R) const { return c < R && wide; }
  __device__ __forceinline__ int slot() const { return s + s0; }    // at or past `wide`: none
  __device__ __forceinline__ void next() {
    s += lanes;
    if (s >= wide) s = 0, c += step;
  }
};

struct LdsRow {
  int src, full, gone1;     // old row; slots that its tokens fill; those from gone0 to here the window has passed
  int grow0, grow1;         // slots of its room; a partly filled one is `full`, before grow0
  int id;                   // the page of that one, -1 where there is none
  int need, copy;           // new pages of the rows before; the row's copy among all, or -1
};
struct Sets {
  uint32_t* used;
  uint32_t* whole;
  int* before;
  __device__ __forceinline__ bool has(int p) const { return used[p >> 5] >> (p & 31) & 1; }
  __device__ __forceinline__ int rank(int p) const { return before[p >> 5] + __popc(used[p >> 5] & ((1u << (p & 31)) - 1u)); }
};

size_t remap_lds(int64_t new_batch, int64_t words) { return 12 * words + sizeof(LdsRow) * new_batch; }

template <bool WIDE, bool APPLY>
__global__ __launch_bounds__(SCAN_THREADS) void remap_kernel(RemapArgs g, int log_lanes) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int2 lds[SCAN_THREADS / 64];
  __shared__ int done;
  const int tid = threadIdx.x, R = g.new_batch, pages = (int)g.pages, words = (int)g.words;
  LdsRow* const rows = (LdsRow*)smem;
  const Sets set = {(uint32_t*)(rows + R), (uint32_t*)(rows + R) + words, (int*)(rows + R) + 2 * words};
  for (int i = tid; i < words; i += SCAN_THREADS) set.used[i] = set.whole[i] = 0;
  if (tid == 0) done = 0;
  for (int c = tid; c < R; c += SCAN_THREADS) {
    const Row w = find_row(g, c);
    const int id = w.part >= 0 ? kept(g, w, w.part) : -1;
    if (id >= 0) put(g.owner + id, 0x7fffffff);
    // slot s is passed when (s + 1) page - 1 <= len - window
    const int64_t passed = g.window ? (int64_t)w.len - g.window + 1 : 0;
    rows[c] = {w.row, w.len >> g.shift, passed > 0 ? (int)(passed >> g.shift) : 0, w.grow0, w.grow1, id, 0, 0};
    put(g.lens_out + c, w.len);
  }
  __syncthreads();

  // the page of slot s of row c, where its tokens fill it and it is kept: no branches, so that the loads do not wait
  // for each other; what is not there is read at the first entry (of any array, where the table has none)
  const int gone0 = (int)min((g.sinks + g.page - 1) >> g.shift, (int64_t)0x7fffffff);
  const int32_t* const table = g.batch && g.width ? g.table : g.counts;
  auto entry = [&](int c, int s) __attribute__((always_inline)) {
    const LdsRow& r = rows[min(c, R - 1)];
    int src = r.src, full = r.full, gone1 = r.gone1;
    if (WIDE) {
      src = __builtin_amdgcn_readfirstlane(src);
      full = __builtin_amdgcn_readfirstlane(full);
      gone1 = __builtin_amdgcn_readfirstlane(gone1);
    }
    const bool go = (c < R) & (s < full) & ((s < gone0) | (s >= gone1));
    const int id = table[go ? (int64_t)src * g.width + s : 0];
    return (go & (id >= 0) & (id < pages)) ? id : -1;
  };
  for (int c = tid; c < R; c += SCAN_THREADS) {
    const int id = rows[c].id;
    if (id < 0) continue;
    atomicOr(&set.used[id >> 5], 1u << (id & 31));
    __hip_atomic_fetch_min(g.owner + id, c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  const int slots = (int)min(g.width, g.width_out), wide = (int)g.width_out;
  for (Walk<WIDE> w(slots, log_lanes); w.any(R);) {
    int id[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k, w.next()) id[k] = entry(w.c, w.slot());
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (id[k] < 0) continue;
      atomicOr(&set.used[id[k] >> 5], 1u << (id[k] & 31));
      atomicOr(&set.whole[id[k] >> 5], 1u << (id[k] & 31));
    }
  }
  __syncthreads();

  int2 total, run = {0, 0};
  for (int b = 0; b < words; b += SCAN_THREADS) {
    const int i = b + tid;
    const int2 mine = {i < words ? __popc(set.used[i]) : 0, 0};
    const int2 at = scan2(mine, lds, &total);
    if (i < words) set.before[i] = run.x + at.x;
    run.x += total.x;
  }
  __syncthreads();                                           // without rows no other one follows before the counts are read
  const int used = run.x;
  run = {0, 0};
  for (int b = 0; b < R; b += SCAN_THREADS) {
    const int c = b + tid;
    int2 mine = {0, 0};
    if (c < R) {
      const LdsRow& r = rows[c];
      mine.y = r.id >= 0 && ((set.whole[r.id >> 5] >> (r.id & 31) & 1) || get(g.owner + r.id) != c);
      mine.x = mine.y + r.grow1 - r.grow0;
    }
    const int2 at = scan2(mine, lds, &total);
    if (c < R) {
      rows[c].need = run.x + at.x;
      rows[c].copy = mine.y ? run.y + at.y : -1;
    }
    run.x += total.x;
    run.y += total.y;
  }
  const int need = run.x, fresh = min(need, pages - used), n = used + fresh;
  int copies = run.y;
  if (fresh < need) {                                        // those of rows whose turn comes before the free pages run out
    int mine = 0;
    for (int c = tid; c < R; c += SCAN_THREADS) mine += rows[c].copy >= 0 && rows[c].need < fresh;
    if (mine) atomicAdd(&done, mine);
    __syncthreads();
    copies = done;
  }
  const int below = n < pages ? set.rank(n) : used, moves = g.compact ? used - below : 0, pairs = moves + copies;
  for (int p = tid; p < pages; p += SCAN_THREADS) {          // the lowest free pages
    const int at = p - set.rank(p);
    if (at >= moves + fresh) break;                          // free pages before a page never get fewer
    if (!set.has(p)) g.free[at] = p;
  }
  if (tid < 4) g.counts[tid] = tid == 0 ? pairs : tid == 1 ? n : tid == 2 ? need - fresh : moves;
  if (!APPLY) {                                              // what the last step reads
    if (tid == 0) *g.info = {used, fresh, n, moves, pairs};
    for (int c = tid; c < R; c += SCAN_THREADS) {
      g.need[c] = rows[c].need;
      g.copy[c] = rows[c].copy;
    }
    if (moves) {
      for (int i = tid; i < words; i += SCAN_THREADS) {
        g.used[i] = set.used[i];
        g.before[i] = set.before[i];
      }
    }
    return;
  }
  __syncthreads();

  for (Walk<WIDE> w(wide, log_lanes); w.any(R);) {
    Walk<WIDE> v = w;
    int id[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k, w.next()) id[k] = entry(w.c, w.slot());
#pragma unroll
    for (int k = 0; k < BATCH; ++k, v.next()) {
      const int s = v.slot();
      if (v.c >= R || s >= wide) continue;
      const LdsRow& r = rows[v.c];
      int to = id[k];
      if (s >= r.full && s < r.grow1) {                      // the partly filled slot, and the room's
        const bool copy = s < r.grow0 && r.copy >= 0;
        if (s < r.grow0) to = r.id;
        if (copy || s >= r.grow0) {
          const int nth = copy ? r.need : r.need + (r.copy >= 0) + s - r.grow0;
          to = nth < fresh ? g.free[moves + nth] : -1;
          if (copy && to >= 0) {
            g.src[moves + r.copy] = r.id;
            g.dst[moves + r.copy] = to;
          }
        } else if (moves && to >= n) {
          to = g.free[set.rank(to) - below];
        }
      } else if (moves && to >= n) {
        to = g.free[set.rank(to) - below];
      }
      g.table_out[v.c * g.width_out + s] = to;
    }
  }
  if (moves) {
    for (int p = n + tid; p < pages; p += SCAN_THREADS) {
      if (!set.has(p)) continue;
      const int k = set.rank(p) - below;
      g.src[k] = p;
      g.dst[k] = g.free[k];
    }
  }
  for (int64_t i = pairs + tid; i < g.capacity; i += SCAN_THREADS) g.src[i] = g.dst[i] = -1;
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

// One launch up to APPLY_SLOTS slots (4032: 8.4 us, 8.6 in two; 1216: 6.5 and 8.1;
// 8064: 11.0 and 9.0), two up to SCAN_SLOTS (20032: 12.2 us, 15.2 in four; 37800:
// 17.7 and 18.6; 64064: 23.7 and 18.1), four beyond or where the rows and the sets
// do not fit the LDS of ONE_LDS bytes.
constexpr int64_t APPLY_SLOTS = 4096, SCAN_SLOTS = 32768;
constexpr size_t ONE_LDS = 56 << 10;

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
  auto blocks = [&](int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + 255) / 256, 8 * num_cu)); };
  const size_t lds = remap_lds(g.new_batch, g.words);
  if (slots <= SCAN_SLOTS && lds <= ONE_LDS) {
    int log_lanes = 2;
    while (log_lanes < 6 && g.width_out >> log_lanes) ++log_lanes;
    const bool apply = slots <= APPLY_SLOTS;
    if (log_lanes == 6 && apply) remap_kernel<true, true><<<1, SCAN_THREADS, lds, st>>>(g, 6);
    else if (log_lanes == 6) remap_kernel<true, false><<<1, SCAN_THREADS, lds, st>>>(g, 6);
    else if (apply) remap_kernel<false, true><<<1, SCAN_THREADS, lds, st>>>(g, log_lanes);
    else remap_kernel<false, false><<<1, SCAN_THREADS, lds, st>>>(g, log_lanes);
    if (!apply) remap_apply_kernel<<<blocks(std::max(slots, g.pages)), 256, 0, st>>>(g);
    return hipGetLastError();
  }
  remap_clear_kernel<<<blocks(std::max(g.words, (int64_t)g.new_batch)), 256, 0, st>>>(g);
  remap_mark_kernel<<<blocks(slots), 256, 0, st>>>(g);
  remap_scan_kernel<<<1, SCAN_THREADS, 0, st>>>(g);
  remap_apply_kernel<<<blocks(std::max(slots, g.pages)), 256, 0, st>>>(g);
  return hipGetLastError();
}

hipError_t launch_copy_pages(const KvCache& c, const int32_t* src, const int32_t* dst, int pairs, const int32_t* count,
                             int num_cu, hipStream_t st) {
  const int64_t pieces = ((int64_t)c.heads * c.page * c.D + PIECE - 1) / PIECE * 2;
  copy_pages_kernel<<<(unsigned)std::min<int64_t>(pairs * pieces, 8 * num_cu), 256, 0, st>>>(c, src, dst, pairs, count);
  return hipGetLastError();
}

}  // namespace lowbit
