// Arguments of the kernels that work out a new table of pages (pages.hip).
#pragma once
#include "kvcache.h"

namespace lowbit {

struct RemapInfo {
  int used, fresh, n, moves, pairs;
};

struct RemapArgs {
  const int32_t* table;     // [batch][width]
  const int32_t* lens;      // [batch]
  const int32_t* rows;      // nullable [new_batch]
  const int32_t* room;      // nullable [new_batch]
  int64_t width, width_out, pages;
  int batch, new_batch, page, shift, compact;
  int most;                 // tokens that a row of either table holds
  int64_t window, sinks;
  int32_t* table_out;       // [new_batch][width_out]
  int32_t* lens_out;        // [new_batch]
  int32_t* src;             // [capacity]
  int32_t* dst;
  int64_t capacity;
  int32_t* counts;          // [4]
  // workspace
  RemapInfo* info;
  uint32_t* used;           // [words] pages of kept slots
  uint32_t* whole;          // [words] those of slots that are no partly filled last page
  int32_t* before;          // [words] used pages before a word
  int32_t* owner;           // [pages] lowest row of a partly filled last page; set for those only
  int32_t* free;            // [pages] lowest free pages, as many as are taken
  int32_t* need;            // [new_batch] new pages of the rows before
  int32_t* copy;            // [new_batch] the row's copy among all, or -1
  int64_t words;
};

}  // namespace lowbit
