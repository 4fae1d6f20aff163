// Launchers of the attention over caches of 8-bit floating point (arguments
// checked by the entry point).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_fp8.h"

namespace attn {
namespace tree {

constexpr int kKeys = 128;     // keys per tile
constexpr int kMostCols = 8;       // columns (token, head) of a unit of attn_tree_fp8_kernel.cuh
constexpr int kRowsPerUnit = 128;  // and of attn_tree_fp8_rows.cuh, which has them as rows
constexpr int kMinSteps = 4;   // pieces of a cut unit are at least about this long

struct Params {
  CUtensorMap tm_k;    // bytes: (d, Hkv, page_size, num_pages), box d x 1 x min(page_size, 128) x 1
  CUtensorMap tm_v;
  PagedKV8 c;
  const uint16_t* q;   // (total, Hq, d)
  uint16_t* o;
  float* lse;          // (Hq, total)
  const int* cu;       // or null: one token per sequence
  const long long* mask;   // or null: chains
  int4* rec;           // per CTA: the unit whose first piece it ran (sequence, unit, pieces, columns)
  float2* part_ml;     // (log2 of the weights' sum, 1; or -inf, 0: no key) [2 CTAs][columns]
  float* part_o;       // O of a piece [2 CTAs][columns][d]
  int* err;
  unsigned long long timeout_ns;
  int B, Hq, total, max_tokens;
  int group, parts;    // query heads per key/value head; units per key/value head
  int abreast;         // unit groups that walk the line side by side (heads_abreast)
  int cuts;            // the table can hold a unit long enough to be cut
  int fp16;
  float scale_log2;
  float inv_group;
};

// cols: the most columns that a unit of the call has.
cudaError_t launch_d64(const Params& p, int cols, int grid, cudaStream_t stream);
cudaError_t launch_d128(const Params& p, int cols, int grid, cudaStream_t stream);
// Units of up to kRowsPerUnit columns, as rows.
cudaError_t launch_rows_d64(const Params& p, int cols, int grid, cudaStream_t stream);
cudaError_t launch_rows_d128(const Params& p, int cols, int grid, cudaStream_t stream);

}  // namespace tree
}  // namespace attn
