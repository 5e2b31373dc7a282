// Microscaled quantisation: values to E4M3 or E2M1 with one power-of-two scale
// per 32, and back.  The formats and the choice of the scale are in
// mx_device.h.
//
// Both directions move memory: a wavefront reads 16 bytes a lane, forms each
// block's largest magnitude across the 4 (BF16) or 8 (FP32) lanes that hold
// it, and writes the packed bytes.  32000 x 4096 BF16 to E2M1 (332 MB) takes 57 to 65 us,
// back 53 to 59, each called again and again; in turn 75 and 54 us.  E4M3
// (397 MB) 68 to 74 us and 66.  Four places a thread and the scales of a wavefront in one store
// were no faster (63 us, E4M3 74 against 70).
#include "mx_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

constexpr int kThreads = 256;
constexpr int kPer = 2;  // places per thread, their loads in flight together

// A thread takes VE consecutive elements at each of kPer places 256 threads
// apart, their loads in flight together.  A row's K / VE threads are never split inside
// a block of 32, so the lanes of a block are active together.
template <int DT, int VE, int FMT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(MxQuantParams p) {
  const int64_t i0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kThreads * kPer) +
                     threadIdx.x;
  const int64_t per_row = p.K / VE;
  int64_t row[kPer], e[kPer];
  float v[kPer][VE];
#pragma unroll
  for (int n = 0; n < kPer; ++n) {
    const int64_t i = i0 + n * kThreads;
    // rows are taken from 32-bit arithmetic when the count allows it
    if (p.small) {
      const uint32_t r = (uint32_t)i / (uint32_t)per_row;
      row[n] = r;
      e[n] = (int64_t)((uint32_t)i - r * (uint32_t)per_row) * VE;
    } else {
      row[n] = i / per_row;
      e[n] = (i - row[n] * per_row) * VE;
    }
#pragma unroll
    for (int j = 0; j < VE; ++j) v[n][j] = 0.0f;
    if (row[n] >= p.rows) continue;
    if constexpr (DT == 0) {
      const float* x = static_cast<const float*>(p.x) + row[n] * p.ldx + e[n];
      if constexpr (VE == 4) {
        const f32x4_t t = *reinterpret_cast<const f32x4_t*>(x);
        v[n][0] = t[0];
        v[n][1] = t[1];
        v[n][2] = t[2];
        v[n][3] = t[3];
      } else {
        v[n][0] = *x;
      }
    } else {
      const uint16_t* x = static_cast<const uint16_t*>(p.x) + row[n] * p.ldx + e[n];
      if constexpr (VE == 8) {
        const u32x4_t t = *reinterpret_cast<const u32x4_t*>(x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[n][2 * j] = bf16_lo(t[j]);
          v[n][2 * j + 1] = bf16_hi(t[j]);
        }
      } else {
        v[n][0] = from_bf16(*x);
      }
    }
  }
  const int64_t rb = FMT == kMxE4M3 ? p.K : p.K / 2;
#pragma unroll
  for (int n = 0; n < kPer; ++n)
    mx_store_block<FMT, VE>(v[n], e[n], p.q + row[n] * rb, p.scales + row[n] * (p.K / kMxBlock),
                            row[n] < p.rows);
}

constexpr int dequant_per(int dtype) { return dtype == 0 ? 1 : kPer; }

// A thread takes 8 values, a quarter of a block, at each of PER places (two for
// BF16: 32000 x 4096 E2M1 72 -> 64 us; one for FP32, whose 32 bytes a lane keep the
// stores busy: 112 us against 128).
template <int DT, int FMT>
__global__ __launch_bounds__(kThreads) void mx_dequantize_kernel(MxDequantParams p) {
  constexpr int PER = dequant_per(DT);
  const int64_t i0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kThreads * PER) +
                     threadIdx.x;
  uint32_t byte[PER];
  u32x2_t q[PER];
#pragma unroll
  for (int n = 0; n < PER; ++n) {
    const int64_t i = i0 + n * kThreads;
    byte[n] = 0;
    q[n] = u32x2_t{0, 0};
    if (i >= p.n8) continue;
    byte[n] = p.scales[i >> 2];
    if constexpr (FMT == kMxE4M3)
      q[n] = reinterpret_cast<const u32x2_t*>(p.q)[i];
    else
      q[n][0] = reinterpret_cast<const uint32_t*>(p.q)[i];
  }
#pragma unroll
  for (int n = 0; n < PER; ++n) {
    const int64_t i = i0 + n * kThreads;
    if (i >= p.n8) continue;
    const float s = byte[n] == 255u ? __builtin_nanf("") : mx_scale_value(byte[n]);
    float v[8];
    if constexpr (FMT == kMxE4M3) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t c = (q[n][h] >> (8 * j)) & 255u;
          const uint32_t mag = c & 127u;
          // a code's bits, moved to FP32's fields, stand for the value times
          // 2^-120 (bias 127 against 7): denormal codes come out right too
          const float m = __uint_as_float(mag << 20) * 0x1p120f;
          const float x = mag == 127u ? __builtin_nanf("") : m;
          v[4 * h + j] = ((c & 128u) ? -x : x) * s;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t c = (q[n][0] >> (4 * j)) & 15u;
        // bias 127 against 1: the fields stand for the value times 2^-126
        const float m = __uint_as_float((c & 7u) << 22) * 0x1p126f;
        v[j] = ((c & 8u) ? -m : m) * s;
      }
    }
    if constexpr (DT == 0) {
      f32x4_t* o = static_cast<f32x4_t*>(p.out) + 2 * i;
      o[0] = f32x4_t{v[0], v[1], v[2], v[3]};
      o[1] = f32x4_t{v[4], v[5], v[6], v[7]};
    } else {
      static_cast<u32x4_t*>(p.out)[i] =
          u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                  pack_bf16x2(v[6], v[7])};
    }
  }
}

template <int DT, int VE>
hipError_t launch_quant(MxQuantParams p, int fmt, hipStream_t stream) {
  const int64_t n = p.rows * (p.K / VE);
  const int64_t wg = (n + kThreads * kPer - 1) / (kThreads * kPer);
  p.small = wg * kThreads * kPer < ((int64_t)1 << 31);
  if (fmt == kMxE4M3)
    hipLaunchKernelGGL((mx_quantize_kernel<DT, VE, kMxE4M3>), grid2(wg), dim3(kThreads),
                       0, stream, p);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<DT, VE, kMxE2M1>), grid2(wg), dim3(kThreads),
                       0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const MxQuantParams& p, int dtype, int fmt, hipStream_t stream) {
  if (p.rows <= 0) return hipSuccess;
  const int es = dtype == 0 ? 4 : 2;
  const bool vec = (p.ldx * es) % 16 == 0 && reinterpret_cast<uintptr_t>(p.x) % 16 == 0;
  if (dtype == 0)
    return vec ? launch_quant<0, 4>(p, fmt, stream) : launch_quant<0, 1>(p, fmt, stream);
  return vec ? launch_quant<1, 8>(p, fmt, stream) : launch_quant<1, 1>(p, fmt, stream);
}

hipError_t launch_mx_dequantize(MxDequantParams p, int64_t n, int fmt, int dtype,
                                hipStream_t stream) {
  if (n <= 0) return hipSuccess;
  p.n8 = n / 8;
  const int64_t per_wg = kThreads * dequant_per(dtype);
  const int64_t wg = (p.n8 + per_wg - 1) / per_wg;
#define VCE_DEQ(DT, FMT)                                                                     \
  hipLaunchKernelGGL((mx_dequantize_kernel<DT, FMT>), grid2(wg), dim3(kThreads), 0, \
                     stream, p)
  if (dtype == 0) {
    if (fmt == kMxE4M3)
      VCE_DEQ(0, kMxE4M3);
    else
      VCE_DEQ(0, kMxE2M1);
  } else {
    if (fmt == kMxE4M3)
      VCE_DEQ(1, kMxE4M3);
    else
      VCE_DEQ(1, kMxE2M1);
  }
#undef VCE_DEQ
  return hipGetLastError();
}

}  // namespace vce
