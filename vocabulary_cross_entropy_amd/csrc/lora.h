// Parameter blocks and launchers of the low-rank adapters.  Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace vce {

constexpr int kLoraRank = 128;       // largest rank
constexpr int kLoraAdapters = 1024;  // most adapters of a call

struct LoraFwdArgs {
  const uint16_t* x;
  int64_t M, H, V, ldx;
  int n, r;
  const uint16_t* a;  // (n, r, H)
  const uint16_t* b;  // (n, V, r)
  const int32_t* adapter;
  const float* scale;  // (n), optional
  const uint16_t* w;   // (V, H), optional
  const void* base;    // (M, V) of the output's type, optional
  int64_t ldb;
  void* out;
  int64_t ldo;
  int dtype;
};

struct LoraBwdArgs {
  const void* dy;  // (M, V) of `dtype`
  int dtype;
  int64_t M, H, V, ldy, ldx;
  const uint16_t* x;
  int n, r;
  const uint16_t* a;
  const uint16_t* b;
  const int32_t* adapter;
  const float* scale;
  const uint16_t* w;        // optional
  const uint16_t* dx_base;  // (M, H), optional
  uint16_t* dx;             // (M, H), optional
  float* da;                // (n, r, H), optional
  float* db;                // (n, V, r), optional
};

bool lora_size_ok(int64_t M, int64_t H, int64_t V, int64_t n, int64_t r);
size_t lora_forward_bytes(int64_t M, int64_t H, int64_t V, int64_t n, int64_t r);
size_t lora_backward_bytes(int64_t M, int64_t H, int64_t V, int64_t n, int64_t r, int dtype);
hipError_t launch_lora_forward(const LoraFwdArgs& p, char* ws, hipStream_t stream);
hipError_t launch_lora_backward(const LoraBwdArgs& p, char* ws, hipStream_t stream);

}  // namespace vce
