// beam.h -- in-place reordering of beams' states, shared by the entry points
// on plain arrays, the 4-bit cache and a context's own cache.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace mk {

// One array of states: per beam `segments` runs of bytes, of which the
// 16-byte columns [first16, first16 + count16) move.  Without pages
// (page16 = 0) beam b's segment i is at base + slot * stride + i * seg_stride;
// with them its logical page lp of page16 columns is at
// base + page * stride + i * seg_stride, page = table[slot * pps + lp], or
// slot * pps + lp without a table.
struct ReorderState {
  uint8_t* base;
  const int32_t* table;
  size_t stride, seg_stride;
  uint32_t page16, first16, count16;
  int32_t pps, pages, segments;
  int32_t slots;      // 1: slot[b] is beam b's slot, else the beam's own number
  int32_t slot[16];
};

struct ReorderArgs {
  ReorderState state[2];
  const int32_t* parents;   // [n_batch][beams], device
  int32_t n_states, beams;
};

cudaError_t launch_reorder(const ReorderArgs& a, int n_batch, cudaStream_t st);

}  // namespace mk
