// Internal declarations of the rotary positions.
#pragma once

#include "q8_cache.h"

namespace q8 {

constexpr int kRopeTensors = 4;

struct RopeArgs {
  const void *x[kRopeTensors];
  void *out[kRopeTensors];
  int64_t x_stride[kRopeTensors], out_stride[kRopeTensors];  // elements between rows
  int upto[kRopeTensors];  // heads of the tensors up to and with this one
  int heads;               // of all tensors
  const uint64_t *turns;   // [rot / 2], fractions of a turn per position in units of 2^-64
  const int *positions;    // [rows], or null: by the sequences
  Seqs s;                  // its table is not used
  int dim, rot;
  int copy;                // whether the channels past rot have to be copied
  int row0;                // first row of the launch (set by the launcher)
  float amplitude;
  int inverse;
};
hipError_t launch_rope(const RopeArgs &a, RowType type, bool interleaved, hipStream_t stream);

}  // namespace q8
