// Rows of grouped work items: every choice (a token's expert, a token's
// adapter) gets the next row of its group's segment.  Shared by the layout
// calls of the grouped products and the adapter call.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace dg {

constexpr int kMaxLayoutGroups = 1024;   // (and one more with `others`)

struct LayoutParams {
  const int32_t* ids;      // [n] group of each choice, counted from `first`
  int n;                   // choices
  int first, groups;       // ids in [first, first + groups) count
  int align;               // segments start at multiples of this (0: masked, segment g starts at g * max_m)
  int max_m;               // masked: rows per group
  int rows;                // rows there are
  int32_t* layout;         // [rows] group of each row or -1, or nullptr
  int32_t* row_of;         // [n] row of each choice or -1, or nullptr
  int32_t* slot_of;        // [rows] choice of each row or -1
  int32_t* counts;         // [groups] or nullptr: choices per group (masked: at most max_m)
  int others;              // nonzero: choices outside the first groups - 1 ids form the last group
};

// Enqueues the layout kernels; `scratch` may be too small for the workgroups'
// counts (then every workgroup counts all the choices itself, in one launch).
hipError_t launch_layout(const LayoutParams& p, void* scratch, size_t scratch_bytes, hipStream_t stream);

}  // namespace dg
