// The head's product over microscaled operands: out = s X W^T, X (M, K) and
// W (V, K) each E4M3 or E2M1 with a scale per 32 along K, FP32 accumulation.
//
// Two ways to multiply:
//  * kScaled: the scaled matrix instructions (v_mfma_scale_f32_16x16x128), which take
//    the stored values and apply both scales.  They add the eight products of
//    consecutive k before the FP32 sum, each cut off 13 bits below the largest of
//    the eight (measured).  Products of two E2M1 values span 8 bits, so
//    nothing is cut; with an E4M3 operand a cut product is off by at most
//    2^-13 of the largest beside it, which a BF16 result (2^-8) does not show.
//  * kBf16: the operands are widened to BF16 in registers, scale included
//    (exact: 4 significant bits), and multiplied by the BF16 instructions at half
//    the rate.  FP32 results with an E4M3 operand take this one.  Supersteps that
//    hold a scale outside 2^-63 .. 2^64 (or a NaN one) could leave BF16's range
//    and go through the scaled instructions instead.
//
// Operand layout of the scaled instruction (measured): lane l holds row l % 16; with
// g = l / 16 its E2M1 slots 0..31 are k = 32 g .. 32 g + 31, its E4M3 slots
// 0..15 are k = 16 g .. and slots 16..31 k = 64 + 16 g ..; lane group g gives
// the scale of k block g, whichever lanes hold that block.  Which four blocks
// of 32 an instruction sums is free as long as both operands agree: a
// superstep of 512 k takes four instructions, instruction s summing blocks s,
// 4 + s, 8 + s and 12 + s, so that an E2M1 lane's four operands are 64
// contiguous bytes and its four scales one dword.  kBf16 gives block 4 g + s
// to lane group g in either format, eight values of it to each of four
// 16x16x32 instructions.
//
// Few tokens: W is read once and bounds the time.  Each wavefront keeps 64 rows of W
// against 16 NB tokens and reads both straight into registers.
#include <type_traits>

#include "mx_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));
typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kRowsPerWave = 64;     // of W
constexpr int kFrags = kRowsPerWave / 16;
constexpr int kSkinnyThreads = 256;

enum Mode { kScaled, kBf16 };

template <int FMT>
struct Fmt {
  static constexpr int kCode = FMT == kMxE4M3 ? 0 : 4;  // the instruction's format field
  static constexpr int kPieces = FMT == kMxE4M3 ? 2 : 1;  // 16-byte pieces per lane and step
  // bytes per 32 values
  static constexpr int kBlockBytes = FMT == kMxE4M3 ? 32 : 16;
};

// One row's operands of a superstep for one lane: the 16-byte pieces of its
// four steps and their scales.  `row` and `srow` point at the row's values and
// scales; blocks at or past nblk read as zeros with TAIL.
template <int FMT, int MODE, bool TAIL>
struct SuperFrag {
  u32x4_t q[4][Fmt<FMT>::kPieces];
  uint32_t sc;
  __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* srow, int sstep, int g,
                                       int nblk) {
    // halves of two blocks for the scaled instruction's E4M3 layout
    constexpr bool kHalves = FMT == kMxE4M3 && MODE == kScaled;
    const int b0 = sstep * 16;
    if constexpr (TAIL) {
      sc = 0;
#pragma unroll
      for (int s = 0; s < 4; ++s)
        sc |= (b0 + 4 * g + s < nblk ? (uint32_t)srow[b0 + 4 * g + s] : 127u) << (8 * s);
    } else {
      // scale rows are K / 32 bytes: only bytes are aligned
      uint32_t t;
      __builtin_memcpy(&t, srow + b0 + 4 * g, 4);
      sc = t;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int h = 0; h < Fmt<FMT>::kPieces; ++h) {
        const int blk = b0 + s + (kHalves ? 4 * (g / 2) + 8 * h : 4 * g);
        const int off = blk * Fmt<FMT>::kBlockBytes + 16 * (kHalves ? g % 2 : h);
        if (!TAIL || blk < nblk)
          q[s][h] = *reinterpret_cast<const u32x4_t*>(row + off);
        else
          q[s][h] = u32x4_t{0, 0, 0, 0};
      }
    }
  }
  __device__ __forceinline__ i32x8_t operand(int s) const {
    i32x8_t r;
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = (int32_t)q[s][0][j];
    if constexpr (FMT == kMxE4M3) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[4 + j] = (int32_t)q[s][1][j];
    } else {
      // the instruction reads four registers of an E2M1 operand
#pragma unroll
      for (int j = 0; j < 4; ++j) r[4 + j] = 0;
    }
    return r;
  }
  // Not 0 where one of the four scales lies outside 64 .. 191.
  __device__ __forceinline__ uint32_t far() const {
    return ~(sc ^ (sc << 1)) & 0x80808080u;
  }
  // operand(s) from kBf16's layout: an E4M3 lane's pieces come from the lanes
  // that hold blocks g / 2 and 2 + g / 2 of the instruction.
  __device__ __forceinline__ i32x8_t operand_moved(int s, int lane) const {
    if constexpr (FMT == kMxE2M1) return operand(s);
    const int g = lane >> 4, src = (lane & 15) + 16 * (g / 2);
    i32x8_t r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int lo = __shfl((int)q[s][0][j], src + 32 * h, 64);
        const int hi = __shfl((int)q[s][Fmt<FMT>::kPieces - 1][j], src + 32 * h, 64);
        r[4 * h + j] = g % 2 ? hi : lo;
      }
    }
    return r;
  }
  // Values 8 t .. 8 t + 7 of step s's block as BF16, scale applied.
  __device__ __forceinline__ bf16x8_t wide(int s, int t) const {
    const float f = __uint_as_float(((sc >> (8 * s)) & 255u) << 23);
    bf16x2_t r[4];
    if constexpr (FMT == kMxE4M3) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t w = q[s][t / 2][2 * (t % 2) + j];
        r[2 * j] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, false);
        r[2 * j + 1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, f, true);
      }
    } else {
      const uint32_t w = q[s][0][t];
      r[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 0);
      r[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 1);
      r[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 2);
      r[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, f, 3);
    }
    return __builtin_shufflevector(__builtin_shufflevector(r[0], r[1], 0, 1, 2, 3),
                                   __builtin_shufflevector(r[2], r[3], 0, 1, 2, 3), 0, 1, 2, 3,
                                   4, 5, 6, 7);
  }
};

template <int FA, int FB>
__device__ __forceinline__ f32x4_t mfma16(const i32x8_t& a, const i32x8_t& b, const f32x4_t& c,
                                          uint32_t sa, uint32_t sb, int s) {
  constexpr int ca = Fmt<FA>::kCode, cb = Fmt<FB>::kCode;
  switch (s) {  // the byte of the scale registers is an immediate
    case 0:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, ca, cb, 0, sa, 0, sb);
    case 1:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, ca, cb, 1, sa, 1, sb);
    case 2:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, ca, cb, 2, sa, 2, sb);
    default:
      return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, ca, cb, 3, sa, 3, sb);
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* out, int64_t at, const f32x4_t& v, float scale,
                                       int n, bool wide) {
  if constexpr (DT == 0) {
    float* o = static_cast<float*>(out) + at;
    if (wide && n >= 4) {
      *reinterpret_cast<f32x4_t*>(o) = f32x4_t{v[0] * scale, v[1] * scale, v[2] * scale,
                                               v[3] * scale};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) o[j] = v[j] * scale;
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    if (wide && n >= 4) {
      *reinterpret_cast<u32x2_t*>(o) = u32x2_t{pack_bf16x2(v[0] * scale, v[1] * scale),
                                               pack_bf16x2(v[2] * scale, v[3] * scale)};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) o[j] = to_bf16(v[j] * scale);
    }
  }
}

// blockIdx.x: 256 rows of W (64 per wavefront), blockIdx.y: 16 NB tokens.
template <int FX, int FW, int MODE, int NB, int DT>
__global__ __launch_bounds__(kSkinnyThreads, 2) void mx_skinny_kernel(MxGemmParams p) {
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int64_t v0 = (int64_t)blockIdx.x * (kRowsPerWave * 4) + wave * kRowsPerWave;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * NB);
  if (v0 >= p.V) return;
  const int nblk = (int)(p.K / kMxBlock);
  const int64_t wb = (int64_t)nblk * Fmt<FW>::kBlockBytes, xb = (int64_t)nblk * Fmt<FX>::kBlockBytes;
  const uint8_t *wr[kFrags], *ws[kFrags], *xr[NB], *xs[NB];
#pragma unroll
  for (int i = 0; i < kFrags; ++i) {  // rows past the end repeat the last one
    const int64_t r = min(v0 + 16 * i + c, p.V - 1);
    wr[i] = p.w + r * wb;
    ws[i] = p.ws + r * nblk;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int64_t r = min(m0 + 16 * i + c, p.M - 1);
    xr[i] = p.x + r * xb;
    xs[i] = p.xs + r * nblk;
  }
  f32x4_t acc[kFrags][NB];
#pragma unroll
  for (int i = 0; i < kFrags; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto step = [&](auto tail, int ss) {
    constexpr bool TAIL = decltype(tail)::value;
    SuperFrag<FW, MODE, TAIL> w[kFrags];
    SuperFrag<FX, MODE, TAIL> x[NB];
#pragma unroll
    for (int i = 0; i < kFrags; ++i) w[i].load(wr[i], ws[i], ss, g, nblk);
#pragma unroll
    for (int j = 0; j < NB; ++j) x[j].load(xr[j], xs[j], ss, g, nblk);
    if constexpr (MODE == kScaled) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int i = 0; i < kFrags; ++i)
#pragma unroll
          for (int j = 0; j < NB; ++j)
            acc[i][j] = mfma16<FW, FX>(w[i].operand(s), x[j].operand(s), acc[i][j], w[i].sc,
                                       x[j].sc, s);
    } else {
      uint32_t far = 0;
#pragma unroll
      for (int i = 0; i < kFrags; ++i) far |= w[i].far();
#pragma unroll
      for (int j = 0; j < NB; ++j) far |= x[j].far();
      if (__any(far != 0)) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int j = 0; j < NB; ++j) {
            const i32x8_t b = x[j].operand_moved(s, lane);
#pragma unroll
            for (int i = 0; i < kFrags; ++i)
              acc[i][j] = mfma16<FW, FX>(w[i].operand_moved(s, lane), b, acc[i][j], w[i].sc,
                                         x[j].sc, s);
          }
      } else {
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            bf16x8_t b[NB];
#pragma unroll
            for (int j = 0; j < NB; ++j) b[j] = x[j].wide(s, t);
#pragma unroll
            for (int i = 0; i < kFrags; ++i) {
              const bf16x8_t a = w[i].wide(s, t);
#pragma unroll
              for (int j = 0; j < NB; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[j], acc[i][j], 0, 0, 0);
            }
          }
      }
    }
  };
  const int full = nblk / 16;
  for (int ss = 0; ss < full; ++ss) step(std::false_type{}, ss);
  if (nblk % 16) step(std::true_type{}, full);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int64_t m = m0 + 16 * j + c;
    if (m >= p.M) continue;
#pragma unroll
    for (int i = 0; i < kFrags; ++i) {
      const int64_t v = v0 + 16 * i + 4 * g;
      const int64_t n = p.V - v;
      if (n > 0) store4<DT>(p.out, m * p.ldo + v, acc[i][j], p.scale, n < 4 ? (int)n : 4, p.wide);
    }
  }
}

template <int FX, int FW, int DT>
hipError_t launch_skinny(const MxGemmParams& p, hipStream_t stream) {
  constexpr int MODE = DT == 0 && (FX == kMxE4M3 || FW == kMxE4M3) ? kBf16 : kScaled;
  const unsigned gx = (unsigned)((p.V + 4 * kRowsPerWave - 1) / (4 * kRowsPerWave));
#define VCE_SKINNY(NB)                                                                      \
  hipLaunchKernelGGL((mx_skinny_kernel<FX, FW, MODE, NB, DT>),                                    \
                     dim3(gx, (unsigned)((p.M + 16 * NB - 1) / (16 * NB))),                 \
                     dim3(kSkinnyThreads), 0, stream, p)
  if (p.M <= 16)
    VCE_SKINNY(1);
  else if (p.M <= 32)
    VCE_SKINNY(2);
  else
    VCE_SKINNY(4);
#undef VCE_SKINNY
  return hipGetLastError();
}

template <int FX, int FW>
hipError_t launch_fmt(const MxGemmParams& p, int dtype, hipStream_t stream) {
  return dtype == 0 ? launch_skinny<FX, FW, 0>(p, stream) : launch_skinny<FX, FW, 1>(p, stream);
}

}  // namespace

hipError_t launch_mx_logits(MxGemmParams p, int x_format, int w_format, int dtype,
                            hipStream_t stream) {
  if (p.M <= 0 || p.V <= 0) return hipSuccess;
  const int n = dtype == 0 ? 16 : 8;  // bytes of four logits
  p.wide = p.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % n == 0;
  if (x_format == kMxE4M3)
    return w_format == kMxE4M3 ? launch_fmt<kMxE4M3, kMxE4M3>(p, dtype, stream)
                               : launch_fmt<kMxE4M3, kMxE2M1>(p, dtype, stream);
  return w_format == kMxE4M3 ? launch_fmt<kMxE2M1, kMxE4M3>(p, dtype, stream)
                             : launch_fmt<kMxE2M1, kMxE2M1>(p, dtype, stream);
}

}  // namespace vce
