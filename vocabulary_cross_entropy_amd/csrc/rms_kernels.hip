// Residual + root-mean-square norm around the vocabulary head.
//
//   h = x + residual,  r = 1 / sqrt(mean_j h_j^2 + eps),  y_j = h_j r (w_j + w0)
// and, for dy and the residual stream's own gradient dh,
//   g_j = dy_j (w_j + w0),  xh_j = h_j r
//   dx_j = r (g_j - xh_j mean_i(g_i xh_i)) + dh_j,   dw_j = sum_rows dy_j xh_j
//
// All of it is bound by memory traffic: a row is read once, held in registers
// as FP32 between the sum of squares and the output, and written once.  A row
// belongs to TPR threads of EPL elements each: a wavefront, or a workgroup of 256
// or 1024 (see pick_shape).  Measured at 16384 x 2304 BF16 with a residual (302 MB either
// way): forward 47 us, 6.4 TB/s; backward 64 us, 4.8 TB/s, and 5 us more for dw's shares.
// The backward takes 225 registers at 40 elements a lane, two wavefronts a SIMD: three packed
// rows and dw are 100 of them, the rest unpacked values kept from one use to the next; held to
// 168 registers it spilled and took 170 us.  Its workgroups of 1024 threads are held to 128
// registers, and where a lane has 32 elements (rows above 16384) or 16 read one by one (odd
// rows above 8192) 27 to 178 of them spill: 2048 x 32768 BF16 319 us, 2048 x 17024 254, 4096
// x 9001 271, 2048 x 16385 797, against 45 to 89 of memory traffic.
//
// Loads go through buffer descriptors that end at the row (a lane past it
// reads zeros), so all loads of a row issue together, without branches.
#include "mx_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

constexpr int kMaxWidth = 32768;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void* p, int bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  void* q = reinterpret_cast<void*>(((uint64_t)hi << 32) | lo);
  return __builtin_amdgcn_make_buffer_rsrc(q, (short)0, __builtin_amdgcn_readfirstlane(bytes),
                                           0x00020000);
}

// VE consecutive elements of a row as stored (VE = 1: one element).
template <int DT, int VE>
struct Raw {
  static constexpr int kWords = DT == 0 ? VE : (VE + 1) / 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rs, int e) {
    if constexpr (VE == 1) {
      if constexpr (DT == 0)
        w[0] = __builtin_amdgcn_raw_buffer_load_b32(rs, e * 4, 0, 0);
      else
        w[0] = __builtin_amdgcn_raw_buffer_load_b16(rs, e * 2, 0, 0);
    } else {
      constexpr int kBytes = DT == 0 ? 4 : 2;
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const u32x4_t t = __builtin_bit_cast(
            u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, e * kBytes + i * 4, 0, 0));
        w[i] = t[0];
        w[i + 1] = t[1];
        w[i + 2] = t[2];
        w[i + 3] = t[3];
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (DT == 0) return __uint_as_float(w[i]);
    if constexpr (VE == 1) return __uint_as_float(w[0] << 16);
    return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};

// The norm's weight, of either type whatever the rows' is.
template <int VE>
__device__ __forceinline__ void load_weight(__amdgpu_buffer_rsrc_t rs, int wdtype, int e,
                                            float* w) {
  if (wdtype == 0) {
    Raw<0, VE> t;
    t.load(rs, e);
#pragma unroll
    for (int i = 0; i < VE; ++i) w[i] = t.get(i);
  } else if constexpr (VE == 4) {
    const u32x2_t t =
        __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(rs, e * 2, 0, 0));
    w[0] = bf16_lo(t[0]);
    w[1] = bf16_hi(t[0]);
    w[2] = bf16_lo(t[1]);
    w[3] = bf16_hi(t[1]);
  } else {
    Raw<1, VE> t;
    t.load(rs, e);
#pragma unroll
    for (int i = 0; i < VE; ++i) w[i] = t.get(i);
  }
}

// Stores VE elements rounded to nearest even.
template <int DT, int VE>
__device__ __forceinline__ void store_elems(void* row, int e, const float* v) {
  if constexpr (DT == 0) {
    float* p = static_cast<float*>(row) + e;
    if constexpr (VE == 1)
      *p = v[0];
    else
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{v[0], v[1], v[2], v[3]};
  } else {
    uint16_t* p = static_cast<uint16_t*>(row) + e;
    if constexpr (VE == 1)
      *p = to_bf16(v[0]);
    else
      *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                               pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  }
}

// Sum over the TPR threads of a row, in a fixed order, given to all of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = s;
    __syncthreads();
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) s += sh[i];
    __syncthreads();
  }
  return s;
}

template <int DT, int VE, int TPR, int EPL, bool MX>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_fwd_kernel(RmsFwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRows = kThreads / TPR;  // rows per workgroup
  constexpr int NV = EPL / VE;
  constexpr int kBytes = DT == 0 ? 4 : 2;
  __shared__ float sh[TPR > 64 ? TPR / 64 : 1];
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows +
                      __builtin_amdgcn_readfirstlane((int)(threadIdx.x / TPR));
  if (row >= p.M) return;  // whole wavefronts; a row of several has its workgroup to itself
  const int t = threadIdx.x % TPR;
  const int H = p.H;
  const char* xr = static_cast<const char*>(p.x) + row * p.ldx * kBytes;
  const __amdgpu_buffer_rsrc_t rx = rsrc_of(xr, H * kBytes);
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(p.weight, H * (p.wdtype == 0 ? 4 : 2));
  float v[NV][VE];
  float ss = 0.0f;
  {
    Raw<DT, VE> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i].load(rx, (i * TPR + t) * VE);
    if (p.residual) {
      const char* rr = static_cast<const char*>(p.residual) + row * p.ldr * kBytes;
      const __amdgpu_buffer_rsrc_t rres = rsrc_of(rr, H * kBytes);
      Raw<DT, VE> res[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) res[i].load(rres, (i * TPR + t) * VE);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j) v[i][j] = raw[i].get(j) + res[i].get(j);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VE; ++j) v[i][j] = raw[i].get(j);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VE; ++j) ss = __builtin_fmaf(v[i][j], v[i][j], ss);
  ss = row_sum<TPR>(ss, sh);
  const float rstd = 1.0f / sqrtf(ss / (float)H + p.eps);
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
  if (p.h) {
    char* hr = static_cast<char*>(p.h) + row * H * kBytes;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VE;
      if (e < H) store_elems<DT, VE>(hr, e, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VE;
    float w[VE], y[VE];
    load_weight<VE>(rw, p.wdtype, e, w);
    // the sum is normed as FP32, before h is rounded for storage
#pragma unroll
    for (int j = 0; j < VE; ++j) y[j] = v[i][j] * rstd * (w[j] + p.w0);
    if constexpr (MX) {
      mx_store_block<kMxE4M3, VE>(y, e, p.q + row * H, p.scales + row * (H / kMxBlock), e < H);
    } else {
      if (e < H) store_elems<DT, VE>(static_cast<char*>(p.y) + row * H * kBytes, e, y);
    }
  }
}

// Each workgroup walks the rows blockIdx.x * kRows + k * gridDim.x * kRows and
// keeps its share of dw in registers (a thread meets the same columns in every
// row); the shares of the workgroup's wavefronts meet in LDS at the end and
// those of the workgroups in rms_dw_kernel, both in a fixed order.
template <int DT, int VE, int TPR, int EPL>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_bwd_kernel(RmsBwdParams p) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kRows = kThreads / TPR;
  constexpr int NV = EPL / VE;
  constexpr int kBytes = DT == 0 ? 4 : 2;
  __shared__ float sh[TPR > 64 ? TPR / 64 : kRows * 64 * VE];
  const int t = threadIdx.x % TPR;
  const int sub = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / TPR));
  const int H = p.H;
  const int rowb = H * kBytes;
  const __amdgpu_buffer_rsrc_t rw = rsrc_of(p.weight, H * (p.wdtype == 0 ? 4 : 2));
  const float invh = 1.0f / (float)H;
  float dw[NV][VE];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VE; ++j) dw[i][j] = 0.0f;
  for (int64_t row = (int64_t)blockIdx.x * kRows + sub; row < p.M;
       row += (int64_t)gridDim.x * kRows) {
    const __amdgpu_buffer_rsrc_t rdy =
        rsrc_of(static_cast<const char*>(p.dy) + row * rowb, rowb);
    const __amdgpu_buffer_rsrc_t rh = rsrc_of(static_cast<const char*>(p.h) + row * rowb, rowb);
    Raw<DT, VE> dy[NV], h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      dy[i].load(rdy, (i * TPR + t) * VE);
      h[i].load(rh, (i * TPR + t) * VE);
    }
    // with the others, not behind the sum: one wait for memory per row (95.9 -> 78.2 us
    // at 16384 x 2304 BF16)
    Raw<DT, VE> dh[NV];
    if (p.dh) {
      const __amdgpu_buffer_rsrc_t rdh = rsrc_of(static_cast<const char*>(p.dh) + row * rowb, rowb);
#pragma unroll
      for (int i = 0; i < NV; ++i) dh[i].load(rdh, (i * TPR + t) * VE);
    }
    const float rstd = p.rstd[row];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[VE];
      load_weight<VE>(rw, p.wdtype, (i * TPR + t) * VE, w);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float xh = h[i].get(j) * rstd;
        const float d = dy[i].get(j);
        dw[i][j] = __builtin_fmaf(d, xh, dw[i][j]);
        dot = __builtin_fmaf(d * (w[j] + p.w0), xh, dot);
      }
    }
    dot = row_sum<TPR>(dot, sh) * invh;
    char* dxr = static_cast<char*>(p.dx) + row * rowb;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VE;
      float w[VE], dx[VE];
      load_weight<VE>(rw, p.wdtype, e, w);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float g = dy[i].get(j) * (w[j] + p.w0);
        dx[j] = rstd * __builtin_fmaf(-(h[i].get(j) * rstd), dot, g);
        if (p.dh) dx[j] += dh[i].get(j);
      }
      if (e < H) store_elems<DT, VE>(dxr, e, dx);
    }
  }
  if (!p.partial) return;
  float* part = p.partial + (int64_t)blockIdx.x * rms_share_width(H);
  if constexpr (TPR > 64) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VE;
      if (e < H)
#pragma unroll
        for (int j = 0; j < VE; ++j) part[e + j] = dw[i][j];
    }
  } else {
    // one vector of every wavefront's share at a time; wavefront 0 adds them
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < VE; ++j) sh[(sub * VE + j) * 64 + t] = dw[i][j];
      __syncthreads();
      const int e = (i * 64 + t) * VE;
      if (sub == 0 && e < H) {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          float s = 0.0f;
#pragma unroll
          for (int k = 0; k < kRows; ++k) s += sh[(k * VE + j) * 64 + t];
          part[e + j] = s;
        }
      }
    }
  }
}

// dw = sum of the workgroups' shares (n_part rows), 32 columns per workgroup (a cache line
// of each share: backward of 1024 x 4096 BF16 17.4 -> 14.0 us against 16), the
// shares dealt over its 32 groups of 32 lanes and added in a fixed order.
__global__ __launch_bounds__(1024) void rms_dw_kernel(const float* partial, int n_part, int H,
                                                      float* dw) {
  __shared__ float sh[32][32];
  const int col = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + col;
  float s = 0.0f;
  if (c < H) {
    // 16 loads in flight, whatever the number of shares
    constexpr int kLoads = 16;
    for (int k0 = grp; k0 < n_part; k0 += 32 * kLoads) {
      float v[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = min(k0 + 32 * i, n_part - 1);
        v[i] = partial[(int64_t)k * rms_share_width(H) + c];
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) s += k0 + 32 * i < n_part ? v[i] : 0.0f;
    }
  }
  sh[grp][col] = s;
  __syncthreads();
  if (threadIdx.x < 32 && c < H) {
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += sh[k][col];
    dw[c] = s;
  }
}

bool vec_ok(int64_t H, int es, int64_t ld) {
  return (H * es) % 16 == 0 && (ld * es) % 16 == 0;
}
bool al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Calls f with the threads per row and elements per lane as constants.  A
// wavefront per row needs no barrier and wins while it holds 16 elements a lane at
// most (forward at H = 1024: 40 us against 45 by 256 threads; at 2304 55 against
// 51); the backward, whose rows meet no other barrier, up to 40 (16384 rows of BF16, calls
// with dw, against 256 threads: H = 1056 41 us and 49, 1536 46 and 50, 2048 57 and 61, 2304
// 68 and 86, 2560 77 and 90; at 4096 with 64 elements 159 against 101).  Rows read one by
// one take 10 elements a lane up to 2560 (against 16: 8192 x 1029 FP32 backward 34 us and
// 54, 1537 40 and 61, 2559 73 and 100; 16384 x 2305 BF16 forward 75 and 90, backward 103
// and 206).  Few rows take more threads each whatever H is.
template <int VE, bool BWD, class F>
hipError_t pick_shape(int64_t M, int H, F f) {
  using std::integral_constant;
#define VCE_SHAPE(T, E) f(integral_constant<int, T>{}, integral_constant<int, E>{})
  if constexpr (VE == 1) {
    if (H <= 1024) return VCE_SHAPE(256, 4);
    if (H <= 2560) return VCE_SHAPE(256, 10);
    if (H <= 4096) return VCE_SHAPE(256, 16);
    if (H <= 8192) return VCE_SHAPE(1024, 8);
    if (H <= 16384) return VCE_SHAPE(1024, 16);
    return VCE_SHAPE(1024, 32);
  } else {
    if (H > 16384) return VCE_SHAPE(1024, 32);
    if (H > 8192) return VCE_SHAPE(1024, 16);
    if (H > 4096) return VCE_SHAPE(256, 32);
    if (H <= 512) return VCE_SHAPE(64, 8);
    if (M >= 1024) {
      if (H <= 1024) return VCE_SHAPE(64, 16);
      if constexpr (BWD)
        if (H <= 2560) return VCE_SHAPE(64, 40);
    }
    return H <= 2048 ? VCE_SHAPE(256, 8) : VCE_SHAPE(256, 16);
  }
#undef VCE_SHAPE
}

template <int DT, int VE, bool MX>
hipError_t launch_fwd(const RmsFwdParams& p, hipStream_t stream) {
  return pick_shape<VE, false>(p.M, p.H, [&](auto tpr, auto epl) {
    constexpr int T = decltype(tpr)::value, E = decltype(epl)::value;
    constexpr int threads = T < 256 ? 256 : T;
    constexpr int rows = threads / T;
    hipLaunchKernelGGL((rms_fwd_kernel<DT, VE, T, E, MX>),
                       grid2((p.M + rows - 1) / rows), dim3(threads), 0, stream, p);
    return hipGetLastError();
  });
}

template <int DT, int VE>
hipError_t launch_bwd(const RmsBwdParams& p, int n_wg, hipStream_t stream) {
  return pick_shape<VE, true>(p.M, p.H, [&](auto tpr, auto epl) {
    constexpr int T = decltype(tpr)::value, E = decltype(epl)::value;
    constexpr int threads = T < 256 ? 256 : T;
    hipLaunchKernelGGL((rms_bwd_kernel<DT, VE, T, E>), dim3((unsigned)n_wg), dim3(threads), 0,
                       stream, p);
    return hipGetLastError();
  });
}

}  // namespace

bool rms_width_ok(int64_t H) { return H >= 1 && H <= kMaxWidth; }

hipError_t launch_rms_forward(const RmsFwdParams& p, int dtype, bool mx, hipStream_t stream) {
  if (p.M <= 0) return hipSuccess;
  const int es = dtype == 0 ? 4 : 2;
  const bool vec = vec_ok(p.H, es, p.ldx) && (!p.residual || vec_ok(p.H, es, p.ldr)) &&
                   al16(p.x) && al16(p.residual) && al16(p.weight) && al16(p.y) && al16(p.h) &&
                   al16(p.q);
  if (dtype == 0) {
    if (mx) return vec ? launch_fwd<0, 4, true>(p, stream) : launch_fwd<0, 1, true>(p, stream);
    return vec ? launch_fwd<0, 4, false>(p, stream) : launch_fwd<0, 1, false>(p, stream);
  }
  if (mx) return vec ? launch_fwd<1, 8, true>(p, stream) : launch_fwd<1, 1, true>(p, stream);
  return vec ? launch_fwd<1, 8, false>(p, stream) : launch_fwd<1, 1, false>(p, stream);
}

// Workgroups of the backward, and so shares of dw: two per CU, four where rows
// are short or read element by element (at 16384 x 2305 BF16 137 -> 103 us), fewer
// where a workgroup would not have at least two rows (300 x 8192 BF16 18.4 -> 14.8 us
// against four).
static int bwd_parts(int64_t M, int most) {
  const int64_t n = (M + 1) / 2;
  return (int)(n < 1 ? 1 : n > most ? most : n);
}

int rms_bwd_parts(int64_t M) { return bwd_parts(M, 1024); }

hipError_t launch_rms_backward(RmsBwdParams p, int dtype, hipStream_t stream) {
  const int es = dtype == 0 ? 4 : 2;
  const bool vec = vec_ok(p.H, es, p.H) && al16(p.dy) && al16(p.h) && al16(p.dh) && al16(p.dx) &&
                   al16(p.weight);
  const int n = bwd_parts(p.M, !vec || p.H <= 1024 ? 1024 : 512);
  if (p.M > 0) {
    hipError_t e;
    if (dtype == 0)
      e = vec ? launch_bwd<0, 4>(p, n, stream) : launch_bwd<0, 1>(p, n, stream);
    else
      e = vec ? launch_bwd<1, 8>(p, n, stream) : launch_bwd<1, 1>(p, n, stream);
    if (e != hipSuccess) return e;
  }
  if (p.dweight) {
    hipLaunchKernelGGL(rms_dw_kernel, dim3((unsigned)((p.H + 31) / 32)), dim3(1024), 0, stream,
                       p.partial, p.M > 0 ? n : 0, p.H, p.dweight);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace vce
