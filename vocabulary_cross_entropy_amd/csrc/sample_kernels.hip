// A token drawn from each row of logits z, from a given uniform number u:
//   w_i = exp((z_i - m) / T), m the row's maximum
//   top-k: the k tokens largest by (z, lower index first)
//   top-p: of those, the shortest prefix in that order whose mass reaches p of
//          theirs (at least one token)
//   min-p: of those, the tokens with w_i >= min_p
//   token: the first kept i, in index order, whose running sum of kept w
//          exceeds u times the whole.   T = 0: the first maximum.
//
// The answer is an index, so the sums must not depend on how they are split:
// weights are computed in FP64 and rounded once to multiples of 2^-fb (fb = 44
// for V up to 2^18), and everything after is 64-bit integer addition, which
// is associative: LDS atomics, wavefront trees and any order give the same
// bits.  FP64 costs no more than unpacked FP32 on this chip.
//
// No sort: thresholds come from radix selection over order-preserving keys.
// A histogram over the distance m - z (128 bins per octave, 16 octaves) finds
// the bin where the count (top-k) or the mass (top-p) is reached; the
// candidates down to it, or if they are too many those of that bin alone, are
// gathered in LDS, and selection by eight key bits at a time finishes there.
#include <math.h>

#include "vce_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr uint32_t kBinBase = 119u << 7;  // bits of 2^-8 over 2^16: bin 0 lies below
constexpr int kCap = 4096;                // candidates held in LDS
constexpr int kLoads = 4;                 // vectors in flight per thread

typedef unsigned long long u64;

template <int DT>
struct Row {
  static constexpr int VE = DT == 0 ? 4 : 8;
  static constexpr int kKeyBits = DT == 0 ? 32 : 16;
  const char* base;   // the row
  int64_t V;
  int off;            // elements from the 16-byte boundary below the row to it
  int nvec;           // 16-byte vectors that hold a part of the row

  __device__ void init(const void* p, int64_t v) {
    constexpr int es = DT == 0 ? 4 : 2;
    base = static_cast<const char*>(p);
    V = v;
    off = (int)(reinterpret_cast<uintptr_t>(p) % 16) / es;
    nvec = (int)((V + off + VE - 1) / VE);
  }
  // Index of element 0 of vector i (negative by `off` for the first).
  __device__ __forceinline__ int64_t first(int i) const { return (int64_t)i * VE - off; }

  // Vector i; elements outside the row come as -inf, -0 as +0.  The first and
  // last vectors are read element by element where the row does not fill them.
  __device__ __forceinline__ void load(int i, float* z) const {
    const int64_t e = first(i);
    if (e >= 0 && e + VE <= V) {
      unpack(*reinterpret_cast<const u32x4_t*>(base + e * (DT == 0 ? 4 : 2)), z);
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        float t = kNegInf;
        if (e + j >= 0 && e + j < V) {
          if constexpr (DT == 0)
            t = reinterpret_cast<const float*>(base)[e + j];
          else
            t = from_bf16(reinterpret_cast<const uint16_t*>(base)[e + j]);
        }
        z[j] = t + 0.0f;
      }
    }
  }
  static __device__ __forceinline__ void unpack(const u32x4_t& w, float* z) {
    if constexpr (DT == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) z[j] = __uint_as_float(w[j]) + 0.0f;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[2 * j] = bf16_lo(w[j]) + 0.0f;
        z[2 * j + 1] = bf16_hi(w[j]) + 0.0f;
      }
    }
  }
  // Larger logits have larger keys.
  static __device__ __forceinline__ uint32_t key(float z) {
    const uint32_t b = __float_as_uint(z);
    const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
    return k >> (32 - kKeyBits);
  }

  // f(first index, z) for the vectors c0 + t, c0 + t + step, ... below c1.
  template <class F>
  __device__ __forceinline__ void each(int c0, int c1, int t, int step, F f) const {
    const int full0 = off ? 1 : 0;
    const int full1 = (int)((V + off) / VE);  // vectors [full0, full1) lie inside the row
    int i = c0 + t;
    for (; i + (kLoads - 1) * step < c1; i += kLoads * step) {
      if (i >= full0 && i + (kLoads - 1) * step < full1) {
        u32x4_t raw[kLoads];
#pragma unroll
        for (int q = 0; q < kLoads; ++q)
          raw[q] = *reinterpret_cast<const u32x4_t*>(base + first(i + q * step) *
                                                                (DT == 0 ? 4 : 2));
#pragma unroll
        for (int q = 0; q < kLoads; ++q) {
          float z[VE];
          unpack(raw[q], z);
          f(first(i + q * step), z);
        }
      } else {
        for (int q = 0; q < kLoads; ++q) {
          float z[VE];
          load(i + q * step, z);
          f(first(i + q * step), z);
        }
      }
    }
    for (; i < c1; i += step) {
      float z[VE];
      load(i, z);
      f(first(i), z);
    }
  }
};

// Fixed-point weights of one row.
struct Weights {
  float m;
  double c;        // log2(e) / T
  double minp;
  bool hard;       // T = 0, or m infinite: only z = m has weight, all the same
  double magic;    // 2^(52 - fb): a double at least that large ends at 2^-fb
  u64 magic_bits;
  double one;      // 2^fb, the weight of z = m

  // 2^x for x <= 0 by 2^n 2^f, |f| <= 1/2, with 2^f - 1 = f g(f), g the
  // polynomial of degree 9 through 2^f's at ten Chebyshev nodes (relative
  // error 6e-16, and exactly 1 at f = 0).  x below -64 rounds to no weight.
  __device__ __forceinline__ double real(float z) const {
    double x = ((double)z - (double)m) * c;
    x = __builtin_fmax(x, -64.0);
    const double r = x + 0x1.8p52;
    const double f = x - (r - 0x1.8p52);
    double g = 0x1.e5e9f548e5725p-28;
    g = __builtin_fma(g, f, 0x1.b6571de2f2351p-24);
    g = __builtin_fma(g, f, 0x1.62bfe46117445p-20);
    g = __builtin_fma(g, f, 0x1.ffcb76789860fp-17);
    g = __builtin_fma(g, f, 0x1.4309130378460p-13);
    g = __builtin_fma(g, f, 0x1.5d87fe908f88ap-10);
    g = __builtin_fma(g, f, 0x1.3b2ab6fba385fp-7);
    g = __builtin_fma(g, f, 0x1.c6b08d7044119p-5);
    g = __builtin_fma(g, f, 0x1.ebfbdff82c590p-3);
    g = __builtin_fma(g, f, 0x1.62e42fefa39f7p-1);
    const double p = __builtin_fma(g, f, 1.0);
    const u64 n = (u64)__builtin_bit_cast(u64, r) << 52;  // n mod 2^12, in the exponent's place
    return __builtin_bit_cast(double, __builtin_bit_cast(u64, p) + n);
  }
  __device__ __forceinline__ u64 fixed(double w) const {
    return __builtin_bit_cast(u64, w + magic) - magic_bits;
  }
  // The weight of z among all tokens (min-p not applied).
  __device__ __forceinline__ u64 all(float z) const {
    if (hard) return z == m ? (u64)one : 0;
    return fixed(real(z));
  }
  // The same with the tokens below min-p left out.
  __device__ __forceinline__ u64 kept(float z) const {
    if (hard) return z == m ? (u64)one : 0;
    const double w = real(z);
    return w >= minp ? fixed(w) : 0;
  }
};

struct Shared {
  u64 mass[kBins];
  uint32_t count[kBins];
  uint32_t key[kCap];
  uint32_t idx[kCap];
  u64 hist[256];
  u64 wave[kWaves];
  u64 wave2[kWaves];
  u64 out[4];
  uint32_t n;
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int d) {
  return (u64)__shfl_up((unsigned long long)v, d, 64);
}

// Sum over the workgroup, the same in every thread.
__device__ __forceinline__ u64 block_sum(u64 v, Shared& sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += (u64)__shfl_xor((unsigned long long)v, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) v += sh.wave[i];
  return v;
}

// A running sum reaches its target: at least one element, and the sum at or
// (strict) beyond it.
__device__ __forceinline__ bool reached(u64 c, double target, bool strict) {
  return c > 0 && (strict ? (double)c > target : (double)c >= target);
}

struct Sel {
  uint32_t key;  // the key at which the running sum, from the largest key down, reaches the target
  u64 above;     // the sum over larger keys
  u64 at;        // the sum over that key
};

// visit(f) calls f(key, amount) for this thread's elements, keys below
// 2^bits.  If the whole sum does not reach the target, the least key is taken.
template <class Visit>
__device__ Sel radix_select(int bits, double target, bool strict, Shared& sh, Visit visit) {
  uint32_t prefix = 0;
  u64 above = 0, at = 0;
  for (int shift = (bits - 1) / 8 * 8; shift >= 0; shift -= 8) {
    __syncthreads();
    if (threadIdx.x < 256) sh.hist[threadIdx.x] = 0;
    __syncthreads();
    visit([&](uint32_t k, u64 a) {
      if (a != 0 && (shift >= 24 || (k >> (shift + 8)) == prefix))
        atomicAdd(&sh.hist[(k >> shift) & 255u], a);
    });
    __syncthreads();
    if (threadIdx.x < 64) {
      const int lane = threadIdx.x;
      u64 h[4], s = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = sh.hist[255 - 4 * lane - j];
        s += h[j];
      }
      u64 run = s;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const u64 o = shfl_up64(run, d);
        if (lane >= d) run += o;
      }
      const uint64_t hit = __ballot(reached(above + run, target, strict));
      const uint64_t some = __ballot(s != 0);
      // the first lane that reaches it, else the last that holds anything
      const int who = hit ? __builtin_ctzll(hit) : some ? 63 - __builtin_clzll(some) : 63;
      if (lane == who) {
        u64 a = above + run - s;
        int pick = -1, last = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (pick < 0) {
            if (h[j] != 0) last = j;
            if (reached(a + h[j], target, strict))
              pick = j;
            else
              a += h[j];
          }
        }
        if (pick < 0) {  // not reached: the last bin that holds anything
          pick = last;
          a -= h[last];
        }
        sh.out[0] = (u64)(255 - 4 * lane - pick);
        sh.out[1] = a;
        sh.out[2] = h[pick];
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)sh.out[0];
    above = sh.out[1];
    at = sh.out[2];
  }
  return Sel{prefix, above, at};
}

// The first index, in order, at which the running sum of amount(index, z)
// exceeds target(whole sum); V if it never does.  Each wavefront sums a
// sixteenth of the range, the sixteenth that holds the crossing is split
// again, down to one vector per lane.
template <int DT, class Target, class Amount>
__device__ int64_t locate(const Row<DT>& row, Shared& sh, Target target, u64* total,
                          Amount amount) {
  constexpr int VE = Row<DT>::VE;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int c0 = 0, c1 = row.nvec;
  u64 before = 0;
  double goal = 0.0;
  bool first = true;
  while (true) {
    const int chunk = (c1 - c0 + kWaves - 1) / kWaves;
    const int a = min(c0 + wave * chunk, c1), b = min(a + chunk, c1);
    u64 s = 0;
    row.each(a, b, lane, 64, [&](int64_t e, const float* z) {
#pragma unroll
      for (int j = 0; j < VE; ++j) s += amount(e + j, z[j]);
    });
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += (u64)__shfl_xor((unsigned long long)s, off, 64);
    __syncthreads();
    if (lane == 0) sh.wave[wave] = s;
    __syncthreads();
    if (first) {
      u64 all = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) all += sh.wave[i];
      *total = all;
      goal = target(all);
      first = false;
    }
    int w = -1;
    for (int i = 0; i < kWaves; ++i) {
      const u64 t = sh.wave[i];
      if ((double)(before + t) > goal && t != 0) {
        w = i;
        break;
      }
      before += t;
    }
    if (w < 0) return row.V;
    const int na = min(c0 + w * chunk, c1);
    c1 = min(na + chunk, c1);
    c0 = na;
    if (c1 - c0 <= 64) break;
  }
  // one vector per lane of wavefront 0
  __syncthreads();
  if (wave == 0) {
    u64 q[VE], s = 0;
    const int i = c0 + lane;
    if (i < c1) {
      float z[VE];
      row.load(i, z);
      const int64_t e = row.first(i);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        q[j] = amount(e + j, z[j]);
        s += q[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) q[j] = 0;
    }
    u64 run = s;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const u64 o = shfl_up64(run, d);
      if (lane >= d) run += o;
    }
    const uint64_t hit = __ballot(s != 0 && (double)(before + run) > goal);
    const int who = hit ? __builtin_ctzll(hit) : 0;
    if (lane == who) {
      u64 c = before + run - s;
      int64_t idx = row.V;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        c += q[j];
        if (idx == row.V && q[j] != 0 && (double)c > goal) idx = row.first(i) + j;
      }
      sh.out[0] = hit ? (u64)idx : (u64)row.V;
    }
  }
  __syncthreads();
  return (int64_t)sh.out[0];
}

__device__ __forceinline__ uint32_t bin_of(float m, float z) {
  if (z == m) return 0;  // m infinite too
  const uint32_t b = __float_as_uint(m - z) >> 16;
  const uint32_t k = b > kBinBase ? b - kBinBase : 0u;
  return k < kBins - 1 ? k : kBins - 1;
}

// Histogram of the row over bin_of: tokens per bin, and with MASS their weights.
template <int DT, bool MASS>
__device__ void histogram(const Row<DT>& row, const Weights& wt, Shared& sh) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    sh.count[i] = 0;
    sh.mass[i] = 0;
  }
  __syncthreads();
  row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t, const float* z) {
#pragma unroll
    for (int j = 0; j < Row<DT>::VE; ++j) {
      if (z[j] == kNegInf || (wt.hard && z[j] != wt.m)) continue;
      const uint32_t b = bin_of(wt.m, z[j]);
      if constexpr (MASS) {
        const u64 q = wt.all(z[j]);
        if (q != 0) atomicAdd(&sh.mass[b], q);
      }
      atomicAdd(&sh.count[b], 1u);
    }
  });
  __syncthreads();
}

struct BinSel {
  int bin;
  u64 above;       // amount in the bins before it
  uint32_t n_incl; // tokens in the bins up to and with it
  uint32_t n_at;
  u64 total;
};

// The first bin where the running amount (mass or count) reaches
// target(total); the last one if it never does.
template <class Amount, class Target>
__device__ BinSel scan_bins(Shared& sh, Amount amount, Target target) {
  constexpr int kPer = kBins / kThreads;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  u64 s = 0;
  uint32_t n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    s += amount(t * kPer + j);
    n += sh.count[t * kPer + j];
  }
  u64 run = s, cnt = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_up64(run, d), c = shfl_up64(cnt, d);
    if (lane >= d) {
      run += o;
      cnt += c;
    }
  }
  __syncthreads();
  if (lane == 63) {
    sh.wave[wave] = run;
    sh.wave2[wave] = cnt;
  }
  __syncthreads();
  u64 base = 0, nbase = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < wave) {
      base += sh.wave[i];
      nbase += sh.wave2[i];
    }
    total += sh.wave[i];
  }
  const double goal = target(total);
  // exactly one thread's bins hold the crossing: before it not reached, with it reached
  const u64 before = base + run - s, upto = base + run;
  if (t == kThreads - 1) {
    sh.out[0] = kBins - 1;
    sh.out[1] = total - amount(kBins - 1);
    sh.out[2] = nbase + cnt;
    sh.out[3] = sh.count[kBins - 1];
  }
  __syncthreads();
  if (!reached(before, goal, false) && reached(upto, goal, false)) {
    u64 a = before;
    uint64_t c = nbase + cnt - n;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const u64 h = amount(t * kPer + j);
      const uint32_t k = sh.count[t * kPer + j];
      if (!reached(a, goal, false) && reached(a + h, goal, false)) {
        sh.out[0] = t * kPer + j;
        sh.out[1] = a;
        sh.out[2] = c + k;
        sh.out[3] = k;
      }
      a += h;
      c += k;
    }
  }
  __syncthreads();
  BinSel r;
  r.bin = (int)sh.out[0];
  r.above = sh.out[1];
  r.n_incl = (uint32_t)sh.out[2];
  r.n_at = (uint32_t)sh.out[3];
  r.total = total;
  __syncthreads();
  return r;
}

// Gathers the tokens of bins [lo, hi] (at most kCap of them) into LDS, in no order.
template <int DT>
__device__ void gather(const Row<DT>& row, const Weights& wt, Shared& sh, uint32_t lo,
                       uint32_t hi) {
  if (threadIdx.x == 0) sh.n = 0;
  __syncthreads();
  row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t e, const float* z) {
#pragma unroll
    for (int j = 0; j < Row<DT>::VE; ++j) {
      if (z[j] == kNegInf || (wt.hard && z[j] != wt.m)) continue;
      const uint32_t b = bin_of(wt.m, z[j]);
      if (b < lo || b > hi) continue;
      const uint32_t at = atomicAdd(&sh.n, 1u);
      if (at < kCap) {
        sh.key[at] = __float_as_uint(z[j]);
        sh.idx[at] = (uint32_t)(e + j);
      }
    }
  });
  __syncthreads();
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleParams p) {
  __shared__ Shared sh;
  typedef Row<DT> R;
  const int64_t r = blockIdx.x;
  const int64_t i0 = r / p.d1, i1 = r - i0 * p.d1;
  R row;
  row.init(static_cast<const char*>(p.logits) + (i0 * p.ls0 + i1 * p.ls1) * (DT == 0 ? 4 : 2),
           p.V);
  const float T = p.temperature ? p.temperature[r] : 1.0f;
  const float top_p = p.top_p ? p.top_p[r] : 1.0f;
  const float min_p = p.min_p ? p.min_p[r] : 0.0f;
  const int32_t top_k = p.top_k ? p.top_k[r] : 0;
  const float u = p.u[r];
  // written so that a NaN fails
  bool ok = T >= 0.0f && T < __builtin_huge_valf() && u >= 0.0f && u < 1.0f &&
            top_p == top_p && min_p == min_p;

  // the maximum, and whether any logit is NaN
  float m = kNegInf;
  bool nan = false;
  row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t, const float* z) {
#pragma unroll
    for (int j = 0; j < R::VE; ++j) {
      m = fmaxf(m, z[j]);
      nan |= z[j] != z[j];
    }
  });
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = __float_as_uint(m);
  const bool any_nan = __syncthreads_or(nan);
  m = kNegInf;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) m = fmaxf(m, __uint_as_float((uint32_t)sh.wave[i]));
  __syncthreads();
  if (any_nan || m == kNegInf) ok = false;
  if (!ok) {
    if (threadIdx.x == 0) {
      p.token[r] = -1;
      if (p.logprob) p.logprob[r] = __builtin_nanf("");
    }
    return;
  }

  Weights wt;
  wt.m = m;
  wt.hard = T == 0.0f || m == __builtin_huge_valf();
  wt.c = wt.hard ? 1.0 : 1.4426950408889634 / (double)T;
  wt.minp = fminf(min_p, 1.0f);  // the maximum is always kept
  wt.magic = p.magic;
  wt.magic_bits = __builtin_bit_cast(u64, p.magic);
  wt.one = p.one;
  const bool greedy = T == 0.0f;

  bool has_k = !greedy && top_k > 0 && top_k < row.V;
  const bool has_p = !greedy && top_p < 1.0f;

  // kept: key > tau, or key = tau and index <= last (tau 0, last V: everything)
  uint32_t tau = 0;
  int64_t last = row.V;
  bool select = false;   // tau is set
  bool listed = false;   // every kept token is in the list
  uint32_t n_list = 0;
  uint64_t ties = 0;     // tokens of key tau that are kept, in index order

  // f(z, index) over the list, or over the row's tokens of bins [lo, hi]
  auto over = [&](bool list, uint32_t lo, uint32_t hi, auto f) {
    if (list) {
      for (uint32_t i = threadIdx.x; i < n_list; i += kThreads)
        f(__uint_as_float(sh.key[i]), (int64_t)sh.idx[i]);
    } else {
      row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t e, const float* z) {
#pragma unroll
        for (int j = 0; j < R::VE; ++j) {
          if (z[j] == kNegInf || (wt.hard && z[j] != m)) continue;
          const uint32_t b = bin_of(m, z[j]);
          if (b >= lo && b <= hi) f(z[j], e + j);
        }
      });
    }
  };

  u64 mass_k = 0;  // mass of the tokens that top-k keeps
  if (has_k) {
    histogram<DT, false>(row, wt, sh);
    const BinSel b = scan_bins(sh, [&](int i) { return (u64)sh.count[i]; },
                               [&](u64) { return (double)top_k; });
    if (b.total <= (u64)top_k) {
      has_k = false;  // fewer admissible tokens than k
    } else {
      select = true;
      listed = b.n_incl <= kCap;
      const uint32_t lo = listed ? 0 : b.bin, hi = b.bin;
      const bool list = listed || b.n_at <= kCap;
      if (list) {
        gather<DT>(row, wt, sh, lo, hi);
        n_list = min(sh.n, (uint32_t)kCap);
      }
      const u64 base = listed ? 0 : b.above;
      const Sel s = radix_select(R::kKeyBits, (double)((u64)top_k - base), false, sh,
                                 [&](auto f) {
        over(list, lo, hi, [&](float z, int64_t) { f(R::key(z), (u64)1); });
      });
      tau = s.key;
      ties = (u64)top_k - base - s.above;
      if (has_p) {
        u64 v = 0, q_tau = 0;
        if (listed) {
          over(true, lo, hi, [&](float z, int64_t) {
            if (R::key(z) > tau) v += wt.all(z);
          });
        } else {
          row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t, const float* z) {
#pragma unroll
            for (int j = 0; j < R::VE; ++j)
              if (R::key(z[j]) > tau) v += wt.all(z[j]);
          });
        }
        if constexpr (DT == 0)
          q_tau = wt.all(__uint_as_float(tau & 0x80000000u ? tau ^ 0x80000000u : ~tau));
        else
          q_tau = wt.all(__uint_as_float((tau & 0x8000u ? tau ^ 0x8000u : ~tau) << 16));
        mass_k = block_sum(v, sh) + ties * q_tau;
      }
    }
  }
  if (has_p) {
    uint32_t lo = 0, hi = kBins - 1;
    u64 base = 0;
    double goal = 0.0;
    bool list = select && listed;
    if (list) {
      goal = (double)top_p * (double)mass_k;
    } else {
      histogram<DT, true>(row, wt, sh);
      const bool sub = select;
      const BinSel b = scan_bins(sh, [&](int i) { return sh.mass[i]; }, [&](u64 total) {
        return (double)top_p * (double)(sub ? mass_k : total);
      });
      goal = (double)top_p * (double)(select ? mass_k : b.total);
      listed = b.n_incl <= kCap;
      lo = listed ? 0 : b.bin;
      hi = b.bin;
      base = listed ? 0 : b.above;
      list = listed || b.n_at <= kCap;
      if (list) {
        gather<DT>(row, wt, sh, lo, hi);
        n_list = min(sh.n, (uint32_t)kCap);
      }
    }
    const uint32_t tau_k = tau;
    const Sel s = radix_select(R::kKeyBits, goal - (double)base, false, sh, [&](auto f) {
      over(list, lo, hi, [&](float z, int64_t) {
        if (R::key(z) >= tau_k) f(R::key(z), wt.all(z));
      });
    });
    const u64 above = base + s.above;
    // tokens of key tau all weigh the same: as many as reach the goal
    u64 n = 0;
    over(list, lo, hi, [&](float z, int64_t) { n += R::key(z) == s.key; });
    n = block_sum(n, sh);
    if (select && s.key == tau_k) n = n < ties ? n : ties;
    const u64 q = n ? s.at : 0;
    u64 each = 0;
    if constexpr (DT == 0)
      each = wt.all(__uint_as_float(s.key & 0x80000000u ? s.key ^ 0x80000000u : ~s.key));
    else
      each = wt.all(__uint_as_float((s.key & 0x8000u ? s.key ^ 0x8000u : ~s.key) << 16));
    u64 t = 1;
    if (q != 0 && each != 0 && goal > (double)above) {
      t = (u64)((goal - (double)above) / (double)each);
      t = t < 1 ? 1 : t;
      while (t > 1 && (double)(above + (t - 1) * each) >= goal) --t;
      while (t < n && (double)(above + t * each) < goal) ++t;
    }
    ties = t < n ? t : n;
    tau = s.key;
    select = true;
  }
  if (select) {
    // the last tie kept, where not all are
    if (listed) {
      u64 n = 0;
      over(true, 0, 0, [&](float z, int64_t) { n += R::key(z) == tau; });
      n = block_sum(n, sh);
      if (ties < n) {
        const int bits = 64 - __builtin_clzll((u64)row.V);
        const Sel s = radix_select(bits, (double)ties, false, sh, [&](auto f) {
          over(true, 0, 0, [&](float z, int64_t i) {
            if (R::key(z) == tau) f((uint32_t)(row.V - 1 - i), (u64)1);
          });
        });
        last = row.V - 1 - (int64_t)s.key;
      }
    } else {
      u64 n;
      last = locate<DT>(row, sh, [&](u64) { return (double)ties - 0.5; }, &n,
                        [&](int64_t, float z) {
        return (u64)(z != kNegInf && R::key(z) == tau && !(wt.hard && z != m));
      });
    }
  }

  u64 total = 0;
  int64_t token;
  if (select && listed) {
    auto amount = [&](float z, int64_t i) -> u64 {
      const uint32_t k = R::key(z);
      return k > tau || (k == tau && i <= last) ? wt.kept(z) : 0;
    };
    u64 v = 0;
    over(true, 0, 0, [&](float z, int64_t i) { v += amount(z, i); });
    total = block_sum(v, sh);
    const int bits = 64 - __builtin_clzll((u64)row.V);
    const Sel s = radix_select(bits, (double)u * (double)total, true, sh, [&](auto f) {
      over(true, 0, 0, [&](float z, int64_t i) { f((uint32_t)(row.V - 1 - i), amount(z, i)); });
    });
    token = row.V - 1 - (int64_t)s.key;
  } else {
    token = locate<DT>(row, sh, [&](u64 all) { return greedy ? 0.0 : (double)u * (double)all; },
                       &total, [&](int64_t i, float z) -> u64 {
      if (!select) return wt.kept(z);
      const uint32_t k = R::key(z);
      return k > tau || (k == tau && i <= last) ? wt.kept(z) : 0;
    });
  }
  if (threadIdx.x == 0) {
    p.token[r] = token;
    if (p.logprob) {
      float lp = 0.0f;
      if (!greedy) {
        float z;
        if constexpr (DT == 0)
          z = reinterpret_cast<const float*>(row.base)[token];
        else
          z = from_bf16(reinterpret_cast<const uint16_t*>(row.base)[token]);
        const double x = wt.hard ? 0.0 : ((double)z - (double)m) / (double)T;
        lp = (float)(x - log((double)total / p.one));
      }
      p.logprob[r] = lp;
    }
  }
}

}  // namespace

// Bits after the point of a weight: the sum over V of them stays below 2^63.
static int weight_bits(int64_t V) {
  int n = 0;
  while (((int64_t)1 << n) < V) ++n;
  const int fb = 62 - n;
  return fb < 44 ? fb : 44;
}

size_t sample_workspace_bytes(int64_t N, int64_t V) {
  (void)N;
  (void)V;
  return 256;
}

hipError_t launch_sample(SampleParams p, int dtype, int64_t N, void* workspace,
                         hipStream_t stream) {
  (void)workspace;
  if (N <= 0) return hipSuccess;
  const int fb = weight_bits(p.V);
  p.magic = ldexp(1.0, 52 - fb);
  p.one = ldexp(1.0, fb);
  if (dtype == 0)
    hipLaunchKernelGGL((sample_row_kernel<0>), dim3((unsigned)N), dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((sample_row_kernel<1>), dim3((unsigned)N), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace vce
