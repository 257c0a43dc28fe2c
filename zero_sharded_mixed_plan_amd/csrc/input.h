// Declarations shared by the input layer's C ABI (input_abi.cpp) and its kernels
// (input.hip): embedding lookup, embedding gradient, dropout.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "zero_internal.h"

namespace zk {

// q = n / d for 0 <= n < 2^31: (n * m) >> sh with m = ceil(2^sh / d) and
// sh = 31 + ceil(log2 d).  The error of m, below 1, adds n / 2^sh < 1 / d to the
// quotient, which cannot carry it past the next integer; m fits 32 bits because
// d > 2^(sh - 32).
struct FastDiv {
  uint32_t d, m, sh;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t lg = 0;
  while (lg < 31 && (uint32_t(1) << lg) < d) ++lg;
  const uint32_t sh = 31 + lg;
  return FastDiv{d, (uint32_t)(((uint64_t(1) << sh) + d - 1) / d), sh};
}

// One launch's dropout.  thr == 0: none.
struct DropK {
  uint32_t key0, key1, step, site;
  const int64_t* step_dev;
  uint32_t row0;
  uint32_t thr;  // kept <=> 16-bit number >= thr
  float ks;      // multiplier of the kept
};

constexpr int kInThreads = 256;      // threads per workgroup of the streaming kernels here
constexpr int kGroup = 8;            // columns per lane and row: one generator call, 16 bytes of a 16-bit type
constexpr int64_t kMaxUnits = (int64_t(1) << 31) - 1;  // (row, 8-column group) units of one launch
// Workgroups of one launch where their number has no such bound: HIP takes fewer than
// 2^32 threads, and beside the milliseconds of so many another launch costs nothing.
constexpr uint32_t kMaxGroups = 1u << 20;

struct DropoutLaunch {
  const char* x;
  const char* res;  // or null
  char* out;
  const char* x_end;    // ends of what the tensors span, for the accesses near them
  const char* res_end;
  int64_t ld_x, ld_res, ld_out;  // bytes
  uint32_t rows, cols;
  uint32_t units;   // rows * ceil(cols / 8)
  FastDiv groups;   // ceil(cols / 8)
  DropK drop;
};

struct LookupLaunch {
  const char* table;
  const char* pos_table;  // or null
  const char* table_end;
  const char* pos_end;
  const void* ids;        // already advanced to row t0
  const void* pos;        // or null; advanced to row t0
  char* out;              // likewise
  int64_t ld_table, ld_pos, ld_out;  // bytes
  int64_t rows, id0, pos_rows;
  int32_t id64;
  uint32_t n, dim, units;
  FastDiv groups;
  uint32_t t0;            // position of this launch's first row in the call
  FastDiv period;         // of the positions, where pos is null
  float scale;
  DropK drop;
};

// --- gradient ---------------------------------------------------------------
constexpr int kSortThreads = 1024;   // 16 waves, one workgroup per class of ids
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortMinClasses = 256; // one workgroup per CU
constexpr int kSortList = 1024;      // own positions a wave keeps in LDS between its two passes, at most
constexpr int kSortAhead = 8;        // loads of 64 ids in flight per wave
constexpr int kSortKeys = 1024;      // rows of one class at most: a list's entry has 10 bits for the row
// Places of a run that one wave sums: 8, 16 or 32, the most that leave kGradWaves
// waves for the sums (8192 ids, 1600 wide: 16 against 8 with twice the waves, 45.1
// against 48.6 us; 3001 ids, 777 wide: 8 against 16, 22 against 27 us).
constexpr int kMinChunk = 8;
constexpr int kMaxLgChunk = 5;
constexpr int kGradWaves = 4096;
constexpr int64_t kLineRow = 1024;   // bytes of a row from which on whole cache lines are zeroed
// Zeroed by one workgroup, or one row: 8 KiB; 16 to 64 KiB took 37 to 38 us for 8192
// ids into 50257 x 1600 bf16 (36.7) and 330 to 339 for 65536 into 128256 x 4096 (316).
constexpr int kFillBytes = 8192;
// Zeroed beside the sort, whose time grows with the ids: 8192 ids into 50257 x 1600
// bf16 36.7 us, against 42 with none and 39.6 with 8 MiB and 1.5 KiB an id; 65536 into 128256 x
// 4096 316 us against 320.
constexpr int64_t kEarlyBytes = 24 << 20, kEarlyBytesPerId = 1536, kEarlyGroupBytes = 65536;
// One launch instead of three for at most this many ids times slabs of 512 columns
// and this many bytes of gradient, in rows not too many to go through.  Measured
// against three: 64 ids, 256 x 64 fp32 5.8 us (9.0), 1000 ids, 8000 x 512 bf16 9.3
// (13.7), 250 ids, 10000 x 1600 bf16 11.2 (12.7).  Beyond, its 256 workgroups zero too
// slowly (50257 x 1600 bf16 47 us against 30), 400 rows each take 18 us
// (100000 x 8 fp32, against 10), and an id that fills the batch waits for one CU
// (1000 times one id, 512 wide, 23 us against 15; 2500 times 57 against 19).
constexpr uint32_t kOnceIds = 1024;
constexpr int64_t kOnceBytes = 32 << 20;
constexpr uint32_t kOnceKeys = 128;  // rows of one class
constexpr uint32_t kOnceRun = 16;    // ids of a row that one wave sums there
constexpr int kJoinThreads = 512;
constexpr int kJoinGroups = 512;

struct GradLaunch {
  const char* dy;
  const char* dy_end;
  const void* ids;        // null: id of t is t mod period
  char* grad;
  int64_t ld_dy, ld_grad; // bytes
  int64_t id0, rows;
  int32_t id64;
  int32_t accumulate;
  uint32_t n;             // ids
  uint32_t dim;
  float factor;           // scale * ks
  DropK drop;
  // ids given: written by the sort
  uint32_t lg_classes;
  uint32_t keys;          // rows of the largest class
  uint32_t* n_valid;      // ids that have a row
  uint4* order;           // [n_valid] (t, row, index within the row's run, length of the run)
  uint8_t* has;           // [rows] whether the row has an id
  // ids == null: the same by arithmetic.  Ids below long_ids occur
  // div_long.d times, the others div_short.d times.
  uint32_t row_lo, row_hi;  // rows [row_lo, row_hi) have occurrences (row = id - id0)
  uint32_t start_lo;        // place of row_lo's first among all ids
  uint32_t long_ids;
  uint32_t split;           // long_ids * div_long.d
  uint32_t total;           // places of rows [row_lo, row_hi)
  uint32_t period;
  FastDiv div_long, div_short;
  // division of the work
  uint32_t places;        // upper bound of the order's length
  uint32_t longest;       // upper bound of a run's length
  uint32_t list;          // entries of a wave's list in the sort
  uint32_t lg_chunk;
  uint32_t window, windows;  // places whose chunks one wave sums; half a chunk, so that both fit 64 lanes
  uint32_t slabs;         // ceil(dim / 512)
  uint32_t join_places;   // places per workgroup of the join
  uint32_t sum_groups;    // workgroups that sum; the others zero fill_rows rows each
  uint32_t first_group;   // of this launch, among all workgroups that sum and zero, or that join
  uint32_t early_row, early_rows;  // rows from early_row on are zeroed beside the sort, early_rows a workgroup
  uint32_t fill_rows;
  FastDiv fill_units;     // 16-byte units of one row,
  uint32_t fill_align;    // counted from a multiple of this
  float* partial;         // [2 * ceil(places / chunk)][slabs][512], in lane order
};

uint32_t grad_lg_chunk(int64_t n_ids, int64_t dim);

int launch_dropout(const DropoutLaunch& a, zero_dtype_t xt, zero_dtype_t ot, void* stream);
int launch_lookup(const LookupLaunch& a, zero_dtype_t tt, zero_dtype_t ot, void* stream);
int launch_embed_grad(const GradLaunch& a, zero_dtype_t dt, zero_dtype_t gt, void* stream);

}  // namespace zk
