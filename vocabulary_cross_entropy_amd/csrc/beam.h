// Parameter blocks and launchers of beam search.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

struct vce_beam_state;

namespace vce {

constexpr int kBeamMost = 128;      // beams of a request
constexpr int kBeamOutMost = 256;   // candidates returned

struct BeamParams {
  const void* logits;
  int64_t K, V, ls0, ls1;
  const float* scores;
  const uint8_t* ended;  // optional
  int64_t end_token;
  int n_out;
  float* score;
  int32_t* parent;
  int64_t* token;
  // set by the launcher
  double poly[10] = {};
  int segs = 0;                // segments per row
  int64_t n = 0;               // rows times segments
  double* seg_sum = nullptr;   // (rows, segs)
  float* seg_max = nullptr;    // (rows, segs)
  float* group_max = nullptr;  // (rows, segs, groups)
};

constexpr int kBeamTensors = 48;  // of a launch: the table stays below 4 KB of arguments

struct BeamState {
  char* data;
  int64_t inner, outer, stride_outer, stride_beam, stride_batch;  // bytes, but outer
  uint32_t blocks;  // workgroups per batch entry
};

struct BeamTable {
  int n;
  uint32_t first[kBeamTensors];
  BeamState t[kBeamTensors];
};

bool beam_size_ok(int64_t B, int64_t K, int64_t V);
size_t beam_workspace_bytes(int64_t B, int64_t K, int64_t V);
hipError_t launch_beam_step(BeamParams p, int dtype, int64_t B, void* workspace,
                            hipStream_t stream);
hipError_t launch_beam_reorder(const vce_beam_state* states, int64_t count, int64_t B, int64_t K,
                               const int32_t* parent, int64_t stride, hipStream_t stream);

}  // namespace vce
