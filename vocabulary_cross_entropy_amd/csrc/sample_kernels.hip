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
//
// A row is cut into segments of 8192 tokens, 32 to a thread:
//  * sample_max_kernel (rows x segments) reads the logits once: the maximum of every
//    thread's 32 tokens (a group) and of the segment.
//  * sample_mass_kernel (rows x segments), once the row's maximum is known, sums
//    the segment's weights for rows without top-k and min-p, and for rows whose
//    top-p stands alone (or whose top-k is large) adds the segment to the row's
//    histogram over the distance m - z (128 bins per octave, 16 octaves).
//  * sample_pick_kernel (rows) draws.  Candidates are bounded from below first: by
//    the k-th largest group maximum (k groups hold at least k tokens as
//    large), by the histogram's bin where the mass is reached, or by min-p
//    itself; only groups that reach the bound are read again and their
//    candidates gathered in LDS.  Up to 256 are ranked by counting, more go
//    through selection by eight key bits at a time.  A row without filters
//    re-reads the one segment in which its sum crosses u.
//  * rows with more candidates than LDS holds: sample_kept_kernel (rows x
//    segments) sums what their threshold keeps, sample_rest_kernel (rows) draws;
//    those whose threshold itself needs more passes it serves from the row.
// The code that a usual row runs is kept short: a kernel this brief waits for
// its instructions more than for its data (one row of 128256 with all filters took 67 us
// in a kernel of 60 KB, most of it instruction fetch).
//
#include <math.h>

#include <type_traits>

#include "vce_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

constexpr int kThreads = 512;   // of the kernel that reads whole rows
constexpr int kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr uint32_t kBinBase = 119u << 7;  // bits of 2^-8 over 2^16: bin 0 lies below
constexpr int kCap = 4096;                // candidates held in LDS
constexpr int kLoads = 4;                 // vectors in flight per thread
constexpr int kSegThreads = 256;
constexpr int kGroup = 32;                // tokens per thread of a segment
constexpr int kSeg = kSegThreads * kGroup;
constexpr int kSmallK = 1024;             // top-k up to here bounds by group maxima

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

// Fixed-point weights of one row.  The coefficients come as kernel
// arguments, so that they sit in scalar registers and each step of the
// polynomial is one instruction.
struct Weights {
  float m;
  bool inf;        // m is infinite: only z = m has weight, all the same
  double md;       // m as FP64
  double c;        // log2(e) / T
  double minp;
  double magic;    // 2^(52 - fb): a double at least that large ends at 2^-fb
  u64 magic_bits;
  const double* poly;

  // 2^x for x <= 0 by 2^n 2^f, |f| <= 1/2, with 2^f - 1 = f g(f), g the
  // polynomial of degree 8 through (2^f - 1) / f at nine Chebyshev nodes (relative
  // error 4e-14, below the 2^-44 of the rounding, and exactly 1 at f = 0).
  // x below -64 rounds to no weight.  For a finite m.
  __device__ __forceinline__ double real(float z) const {
    double x = ((double)z - md) * c;
    x = __builtin_fmax(x, -64.0);
    const double r = x + 0x1.8p52;
    const double f = x - (r - 0x1.8p52);
    double g = poly[8];
#pragma unroll
    for (int i = 7; i >= 0; --i) g = __builtin_fma(g, f, poly[i]);
    const double p = __builtin_fma(g, f, 1.0);
    // n sits in r's low word; it is added to p's exponent
    const u64 b = __builtin_bit_cast(u64, p);
    const uint32_t n = (uint32_t)__builtin_bit_cast(u64, r);
    const uint32_t hi = (uint32_t)(b >> 32) + (n << 20);
    return __builtin_bit_cast(double, ((u64)hi << 32) | (uint32_t)b);
  }
  __device__ __forceinline__ double weight(float z) const {
    if (inf) return z == m ? 1.0 : 0.0;
    return real(z);
  }
  __device__ __forceinline__ u64 fixed(double w) const {
    return __builtin_bit_cast(u64, w + magic) - magic_bits;
  }
  // The weight of z among all tokens (min-p not applied).
  __device__ __forceinline__ u64 all(float z) const { return fixed(weight(z)); }
  // The same with the tokens below min-p left out.
  __device__ __forceinline__ u64 kept(float z) const {
    const double w = weight(z);
    return w >= minp ? fixed(w) : 0;
  }
};

struct Scratch {
  u64 hist[256];
  u64 wave[kWaves];
  u64 wave2[kWaves];
  u64 out[4];
  uint32_t n;
};

struct Shared : Scratch {
  u64 mass[kBins];
  uint32_t count[kBins];
  uint32_t key[kCap];  // candidates: the logit's bits, its index
  uint32_t idx[kCap];
};

// A candidate: the key of its logit, its index, and its weight, with the top
// bit set unless min-p drops it.
struct alignas(16) Entry {
  uint32_t key, idx;
  u64 q;
};
constexpr u64 kKeptBit = (u64)1 << 63;

constexpr int kGroupBatch = 16;  // segments whose group maxima a thread loads at once

struct PickShared : Scratch {
  Entry list[kCap];
  uint16_t group[kGroupBatch * kSegThreads];
  uint32_t n_groups;
};

__device__ __forceinline__ u64 shfl_up64(u64 v, int d) {
  return (u64)__shfl_up((unsigned long long)v, d, 64);
}

// Sum over the workgroup, the same in every thread.
template <int NW, class S>
__device__ __forceinline__ u64 block_sum(u64 v, S& sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += (u64)__shfl_xor((unsigned long long)v, off, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < NW; ++i) v += sh.wave[i];
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
template <class S, class Visit>
__device__ __forceinline__ Sel radix_select(int bits, double target, bool strict, S& sh,
                                            Visit visit) {
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
          a -= last == 0 ? h[0] : last == 1 ? h[1] : last == 2 ? h[2] : h[3];
        }
        sh.out[0] = (u64)(255 - 4 * lane - pick);
        sh.out[1] = a;
        sh.out[2] = pick == 0 ? h[0] : pick == 1 ? h[1] : pick == 2 ? h[2] : h[3];
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)sh.out[0];
    above = sh.out[1];
    at = sh.out[2];
  }
  return Sel{prefix, above, at};
}

// The first index, in order, of vectors [c0, c1) at which the running sum of
// amount(index, z), from `before` on, exceeds target(sum of the range); V if it
// never does.  Each wavefront sums a
// sixteenth of the range, the sixteenth that holds the crossing is split
// again, down to one vector per lane.
template <int DT, class Target, class Amount>
__device__ __forceinline__ int64_t locate(const Row<DT>& row, int c0, int c1, Shared& sh, u64 before,
                          Target target, u64* total, Amount amount) {
  constexpr int VE = Row<DT>::VE;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
__device__ __forceinline__ void histogram(const Row<DT>& row, const Weights& wt, Shared& sh) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) {
    sh.count[i] = 0;
    sh.mass[i] = 0;
  }
  __syncthreads();
  row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t, const float* z) {
#pragma unroll
    for (int j = 0; j < Row<DT>::VE; ++j) {
      if (z[j] == kNegInf) continue;
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
__device__ __forceinline__ BinSel scan_bins(Shared& sh, Amount amount, Target target) {
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
__device__ __forceinline__ void gather(const Row<DT>& row, const Weights& wt, Shared& sh, uint32_t lo,
                       uint32_t hi) {
  if (threadIdx.x == 0) sh.n = 0;
  __syncthreads();
  row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t e, const float* z) {
#pragma unroll
    for (int j = 0; j < Row<DT>::VE; ++j) {
      if (z[j] == kNegInf) continue;
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

// What a row asks for, from its parameters alone.
struct Ask {
  float T, u;
  double p, minp;
  int32_t k;
  bool ok, greedy, has_k, has_p, has_min;
  // so short a row that all of it is gathered
  __device__ __forceinline__ bool list_all(int64_t V) const { return V <= kCap; }
  // few enough tokens asked for that the group maxima bound them closely
  __device__ __forceinline__ bool group_bound(int64_t V) const {
    return has_k && k <= kSmallK && k <= V / (4 * kGroup);
  }
  // by the histogram: top-p alone, or a top-k too large for the group maxima
  __device__ __forceinline__ bool hist(int64_t V) const {
    return ok && !greedy && !list_all(V) && (has_k ? !group_bound(V) : has_p);
  }
  __device__ __forceinline__ bool plain(int64_t V) const {
    return ok && !greedy && !list_all(V) && !has_k && !has_p && !has_min;
  }
};

__device__ __forceinline__ Ask ask_of(const SampleParams& p, int64_t r) {
  Ask a;
  a.T = p.temperature ? p.temperature[r] : 1.0f;
  const float top_p = p.top_p ? p.top_p[r] : 1.0f;
  const float min_p = p.min_p ? p.min_p[r] : 0.0f;
  a.k = p.top_k ? p.top_k[r] : 0;
  a.u = p.u[r];
  // written so that a NaN fails
  a.ok = a.T >= 0.0f && a.T < __builtin_huge_valf() && a.u >= 0.0f && a.u < 1.0f &&
         top_p == top_p && min_p == min_p;
  a.greedy = a.T == 0.0f;
  a.has_k = a.k > 0 && a.k < p.V;
  a.has_p = top_p < 1.0f;
  a.has_min = min_p > 0.0f;
  a.p = fmaxf(top_p, 0.0f);      // the first token is always kept
  a.minp = fminf(min_p, 1.0f);   // and so are the maxima
  return a;
}

__device__ __forceinline__ Weights weights_of(const SampleParams& p, const Ask& a, float m) {
  Weights wt;
  wt.m = m;
  wt.inf = m == __builtin_huge_valf();
  wt.md = (double)m;
  wt.c = 1.4426950408889634 / (double)a.T;
  wt.minp = a.minp;
  wt.magic = p.magic;
  wt.magic_bits = __builtin_bit_cast(u64, p.magic);
  wt.poly = p.poly;
  return wt;
}

template <int DT>
__device__ __forceinline__ Row<DT> row_of(const SampleParams& p, int64_t r) {
  const int64_t i0 = r / p.d1, i1 = r - i0 * p.d1;
  Row<DT> row;
  row.init(static_cast<const char*>(p.logits) + (i0 * p.ls0 + i1 * p.ls1) * (DT == 0 ? 4 : 2),
           p.V);
  return row;
}

// The row's maximum from its segments' (NaN if any is); whole wavefronts call it.
__device__ __forceinline__ float row_max(const float* seg_max, int n) {
  float m = kNegInf;
  bool nan = false;
  for (int i = threadIdx.x & 63; i < n; i += 64) {
    const float v = seg_max[i];
    nan |= v != v;
    m = fmaxf(m, v);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  return __any(nan) ? __builtin_nanf("") : m;
}

__device__ __forceinline__ u64 wave_sum(u64 v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += (u64)__shfl_xor((unsigned long long)v, off, 64);
  return v;
}

// Running sum over the lanes, each with its own share included.
__device__ __forceinline__ u64 wave_scan(u64 v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const u64 o = shfl_up64(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// The 32 tokens of a thread of a segment: vectors v0, v0 + 256, ... of the row,
// -inf past its ends.
template <int DT>
__device__ __forceinline__ void load_group(const Row<DT>& row, int v0,
                                           float (&z)[kGroup / Row<DT>::VE][Row<DT>::VE]) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  const int last = v0 + (kVec - 1) * kSegThreads;
  if (last < (int)((row.V + row.off) / R::VE) && (v0 > 0 || row.off == 0)) {
    u32x4_t raw[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      raw[j] = *reinterpret_cast<const u32x4_t*>(row.base + row.first(v0 + j * kSegThreads) *
                                                                (DT == 0 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < kVec; ++j) R::unpack(raw[j], z[j]);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      if (v0 + j * kSegThreads < row.nvec) {
        row.load(v0 + j * kSegThreads, z[j]);
      } else {
#pragma unroll
        for (int q = 0; q < R::VE; ++q) z[j][q] = kNegInf;
      }
    }
  }
}

// blockIdx.x: row, blockIdx.y: segment.
template <int DT>
__global__ __launch_bounds__(kSegThreads) void sample_max_kernel(SampleParams p) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  __shared__ float sh[kSegThreads / 64];
  const int64_t r = blockIdx.x;
  const int seg = blockIdx.y, t = threadIdx.x;
  const R row = row_of<DT>(p, r);
  float z[kVec][R::VE];
  load_group<DT>(row, seg * (kSegThreads * kVec) + t, z);
  float m = kNegInf;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kVec; ++j)
#pragma unroll
    for (int q = 0; q < R::VE; ++q) {
      m = fmaxf(m, z[j][q]);
      nan |= z[j][q] != z[j][q];
    }
  p.group_max[(r * p.segs + seg) * kSegThreads + t] = m;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (__any(nan)) m = __builtin_nanf("");
  if ((t & 63) == 0) sh[t >> 6] = m;
  // the row's histogram starts at zero, a share of it per segment
  if (ask_of(p, r).hist(p.V)) {
    for (int64_t b = seg * kSegThreads + t; b < kBins; b += (int64_t)p.segs * kSegThreads) {
      p.hist_mass[r * kBins + b] = 0;
      p.hist_count[r * kBins + b] = 0;
    }
  }
  __syncthreads();
  if (t == 0) {
    bool any = false;
    float s = kNegInf;
#pragma unroll
    for (int i = 0; i < kSegThreads / 64; ++i) {
      any |= sh[i] != sh[i];
      s = fmaxf(s, sh[i]);
    }
    p.seg_max[r * p.segs + seg] = any ? __builtin_nanf("") : s;
  }
}

// For rows without filters the segment's mass; for rows that go by the
// histogram its counts (top-k) or its masses and the whole (top-p).
// Top-p needs no token lighter than q0 = (1 - p) L / V, L a lower bound on
// the row's mass (the sum over the segments' maxima): all such tokens together
// weigh less than (1 - p) of the row, so its p-th part is reached before them.
// They stay out of the histogram, which keeps most LDS atomics away.
template <int DT>
__global__ __launch_bounds__(kSegThreads, 4) void sample_mass_kernel(SampleParams p) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  __shared__ u64 mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ u64 part[kSegThreads / 64];
  const int64_t r = blockIdx.x;
  const int seg = blockIdx.y, t = threadIdx.x;
  const Ask a = ask_of(p, r);
  const bool plain = a.plain(p.V), hist = a.hist(p.V);
  if (!plain && !hist) return;
  const float* seg_max = p.seg_max + r * p.segs;
  const float m = row_max(seg_max, p.segs);
  if (!(m > kNegInf)) return;  // no admissible token, or NaN
  const Weights wt = weights_of(p, a, m);
  const R row = row_of<DT>(p, r);
  float z[kVec][R::VE];
  load_group<DT>(row, seg * (kSegThreads * kVec) + t, z);
  u64 s = 0;
  if (plain) {
    if (wt.inf) {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) s += wt.fixed(z[j / R::VE][j % R::VE] == m ? 1.0 : 0.0);
    } else {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) s += wt.fixed(wt.real(z[j / R::VE][j % R::VE]));
    }
  } else {
    for (int b = t; b < kBins; b += kSegThreads) {
      mass[b] = 0;
      count[b] = 0;
    }
    u64 q0 = 0;
    if (!a.has_k) {
      u64 low = 0;
      for (int i = t & 63; i < p.segs; i += 64) low += wt.all(seg_max[i]);
      q0 = (u64)((1.0 - a.p) * (double)wave_sum(low) / (double)p.V);
    }
    __syncthreads();
    if (wt.inf || a.has_k) {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const float v = z[j / R::VE][j % R::VE];
        const u64 q = a.has_k ? 0 : wt.all(v);
        s += q;
        if (v != kNegInf && q >= q0) {
          atomicAdd(&count[bin_of(m, v)], 1u);
          if (q != 0) atomicAdd(&mass[bin_of(m, v)], q);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const float v = z[j / R::VE][j % R::VE];
        const u64 q = wt.fixed(wt.real(v));
        s += q;
        if (q >= q0 && q != 0) {
          const uint32_t b = bin_of(m, v);
          atomicAdd(&count[b], 1u);
          atomicAdd(&mass[b], q);
        }
      }
    }
  }
  s = wave_sum(s);
  if ((t & 63) == 0) part[t >> 6] = s;
  __syncthreads();
  if (t == 0) p.seg_sum[r * p.segs + seg] = part[0] + part[1] + part[2] + part[3];
  if (hist) {
    for (int b = t; b < kBins; b += kSegThreads) {
      if (count[b]) atomicAdd(&p.hist_count[r * kBins + b], count[b]);
      if (mass[b]) atomicAdd((u64*)&p.hist_mass[r * kBins + b], mass[b]);
    }
  }
}

template <int DT>
__device__ __forceinline__ float key_value(uint32_t k) {
  if constexpr (DT == 0) return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  return __uint_as_float((k & 0x8000u ? k ^ 0x8000u : ~k) << 16);
}

// How many tokens of weight `each` it takes beyond `above` to reach the goal,
// 1 .. n.
__device__ __forceinline__ u64 ties_needed(u64 above, u64 each, u64 n, double goal) {
  u64 t = 1;
  if (each != 0 && goal > (double)above) {
    t = (u64)((goal - (double)above) / (double)each);
    t = t < 1 ? 1 : t;
    while (t > 1 && (double)(above + (t - 1) * each) >= goal) --t;
    while (t < n && (double)(above + t * each) < goal) ++t;
  }
  return t < n ? t : n;
}

// m - z, 0 for z = m also where both are infinite.
__device__ __forceinline__ float distance(float m, float z) { return z == m ? 0.0f : m - z; }

// f(group, maximum) for this thread's groups of segments g0 .. g0 + 15, their
// loads in flight together.
template <class F>
__device__ __forceinline__ void each_group(const float* gm, int segs, int g0, F f) {
  float top[kGroupBatch];
#pragma unroll
  for (int i = 0; i < kGroupBatch; ++i)
    top[i] = g0 + i < segs ? gm[(g0 + i) * kSegThreads + threadIdx.x] : kNegInf;
#pragma unroll
  for (int i = 0; i < kGroupBatch; ++i)
    if (top[i] != kNegInf) f(i * kSegThreads + threadIdx.x, top[i]);
}

// Gathers into LDS the tokens with lo <= m - z <= hi, in no order, from the
// groups whose maximum is within hi: first those groups are listed, then their
// vectors are dealt over the threads, so that all loads wait together.
// Returns the number of tokens; above kCap the list is cut off.
template <int DT>
__device__ __forceinline__ uint32_t gather_groups(const Row<DT>& row, const SampleParams& p,
                                                  int64_t r, const Weights& wt, float lo, float hi,
                                                  PickShared& sh) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  const float* gm = p.group_max + r * p.segs * kSegThreads;
  __syncthreads();
  if (threadIdx.x == 0) sh.n = 0;
  for (int g0 = 0; g0 < p.segs; g0 += kGroupBatch) {
    if (threadIdx.x == 0) sh.n_groups = 0;
    __syncthreads();
    each_group(gm, p.segs, g0, [&](int i, float top) {
      if (distance(wt.m, top) <= hi) sh.group[atomicAdd(&sh.n_groups, 1u)] = (uint16_t)i;
    });
    __syncthreads();
    const int items = (int)sh.n_groups * kVec;
    for (int i = threadIdx.x; i < items; i += kSegThreads) {
      const int g = sh.group[i / kVec];
      const int v = (g0 + g / kSegThreads) * (kSegThreads * kVec) +
                    (i % kVec) * kSegThreads + g % kSegThreads;
      if (v >= row.nvec) continue;
      float z[R::VE];
      row.load(v, z);
      uint32_t in = 0;
#pragma unroll
      for (int q = 0; q < R::VE; ++q) {
        const float d = distance(wt.m, z[q]);
        in |= (z[q] != kNegInf && d >= lo && d <= hi ? 1u : 0u) << q;
      }
      while (in) {
        const int q = __builtin_ctz(in);
        in &= in - 1;
        float x = z[0];
#pragma unroll
        for (int j = 1; j < R::VE; ++j) x = q == j ? z[j] : x;
        const uint32_t at = atomicAdd(&sh.n, 1u);
        if (at < kCap) {
          const double w = wt.weight(x);
          sh.list[at] = Entry{R::key(x), (uint32_t)(row.first(v) + q),
                              wt.fixed(w) | (w >= wt.minp ? kKeptBit : 0)};
        }
      }
    }
    __syncthreads();
  }
  return sh.n;
}

struct Drawn {
  int64_t token;
  u64 total;     // weight of all kept tokens
  // a threshold without a token: kept are the keys above tau, and the first
  // `ties` tokens of key tau
  uint32_t tau;
  u64 ties;
};

// Draws from the list of candidates, which holds every token the filters can
// keep; `mass` is the weight that top-p refers to without top-k.  With
// `threshold` the list holds one bin of the histogram, `above` is the
// weight before it, and only top-p's threshold is taken.
template <int DT>
__device__ __forceinline__ Drawn draw_list(const Ask& a, const Weights& wt, int64_t V, uint32_t n,
                                           u64 mass, bool threshold, u64 above, PickShared& sh) {
  typedef Row<DT> R;
  constexpr int NW = kSegThreads / 64;
  const uint32_t t = threadIdx.x;
  Drawn d;
  d.token = 0;
  d.total = 0;
  d.tau = 0;
  d.ties = 0;
  if (n <= kSegThreads && !threshold) {
    // one candidate per thread: its rank and the weight ranked before it
    const bool mine = t < n;
    const Entry e = mine ? sh.list[t] : Entry{0, 0, 0};
    const u64 q = e.q & ~kKeptBit;
    uint32_t rank = 0;
    u64 before = 0;
    for (uint32_t j = 0; j < n; ++j) {
      const Entry o = sh.list[j];
      if (o.key > e.key || (o.key == e.key && o.idx < e.idx)) {
        ++rank;
        before += o.q & ~kKeptBit;
      }
    }
    bool keep = mine && (!a.has_k || rank < (uint32_t)a.k);
    if (a.has_p) {
      if (a.has_k) mass = block_sum<NW>(keep ? q : 0, sh);
      keep = keep && (rank == 0 || (double)before < a.p * (double)mass);
    }
    keep = keep && (e.q & kKeptBit);
    d.total = block_sum<NW>(keep ? q : 0, sh);  // a barrier: the list has been read
    if (mine) sh.list[t].q = keep ? q : 0;
    if (t == 0) sh.out[0] = 0;
    __syncthreads();
    u64 upto = 0;
    for (uint32_t j = 0; j < n; ++j) {
      const Entry o = sh.list[j];
      if (o.idx <= e.idx) upto += o.q;
    }
    const double goal = (double)a.u * (double)d.total;
    // one kept candidate takes the sum across the goal
    if (keep && q != 0 && (double)upto > goal && !((double)(upto - q) > goal))
      sh.out[0] = e.idx;
    __syncthreads();
    d.token = (int64_t)sh.out[0];
    return d;
  }
  n = n < kCap ? n : kCap;
  u64 ties = ~(u64)0;  // none: no threshold
  uint32_t tau = 0, last = 0xffffffffu;
  const int idx_bits = 64 - __builtin_clzll((u64)V);
  for (int stage = threshold ? 1 : 0; stage < (threshold ? 2 : 4); ++stage) {
    double goal = 0.0;
    if (stage == 0) {  // top-k
      if (!a.has_k || (u64)a.k >= n) continue;
      goal = (double)a.k;
    } else if (stage == 1) {  // top-p
      if (!a.has_p) continue;
      if (a.has_k) {
        u64 v = 0;
        for (uint32_t i = t; i < n; i += kSegThreads)
          if (ties == ~(u64)0 || sh.list[i].key > tau) v += sh.list[i].q & ~kKeptBit;
        mass = block_sum<NW>(v, sh);
        if (ties != ~(u64)0) mass += ties * wt.all(key_value<DT>(tau));
      }
      goal = a.p * (double)mass - (double)above;
    } else if (stage == 2) {  // the last tie kept, where not all are
      if (ties == ~(u64)0) continue;
      u64 c = 0;
      for (uint32_t i = t; i < n; i += kSegThreads) c += sh.list[i].key == tau;
      if (ties >= block_sum<NW>(c, sh)) continue;
      goal = (double)ties;
    } else {  // the token
      u64 v = 0;
      for (uint32_t i = t; i < n; i += kSegThreads) {
        const Entry e = sh.list[i];
        if ((e.q & kKeptBit) && (e.key > tau || (e.key == tau && e.idx <= last)))
          v += e.q & ~kKeptBit;
      }
      d.total = block_sum<NW>(v, sh);
      goal = (double)a.u * (double)d.total;
    }
    const Sel s = radix_select(stage < 2 ? R::kKeyBits : idx_bits, goal, stage == 3, sh,
                               [&](auto f) {
      for (uint32_t i = t; i < n; i += kSegThreads) {
        const Entry e = sh.list[i];
        const bool in = stage == 0   ? true
                        : stage == 1 ? e.key >= tau
                        : stage == 2 ? e.key == tau
                                     : (e.q & kKeptBit) &&
                                           (e.key > tau || (e.key == tau && e.idx <= last));
        const u64 w = stage == 1 || stage == 3 ? e.q & ~kKeptBit : (u64)1;
        if (in) f(stage < 2 ? e.key : (uint32_t)(V - 1 - e.idx), w);
      }
    });
    if (stage == 0) {
      tau = s.key;
      ties = (u64)a.k - s.above;
    } else if (stage == 1) {
      u64 c = 0;
      for (uint32_t i = t; i < n; i += kSegThreads) c += sh.list[i].key == s.key;
      c = block_sum<NW>(c, sh);
      if (s.key == tau && ties < c) c = ties;
      ties = ties_needed(s.above, wt.all(key_value<DT>(s.key)), c, goal);
      tau = s.key;
    } else if (stage == 2) {
      last = (uint32_t)(V - 1 - s.key);
    } else {
      d.token = V - 1 - (int64_t)s.key;
    }
  }
  d.tau = tau;
  d.ties = ties;
  return d;
}

// The token and its log-probability, by one thread.
template <int DT>
__device__ __forceinline__ void write_out(const SampleParams& p, int64_t r, const Row<DT>& row,
                                          const Ask& a, float m, int64_t token, u64 total) {
  p.token[r] = token;
  if (!p.logprob) return;
  float lp = 0.0f;
  if (!a.greedy) {
    float z;
    if constexpr (DT == 0)
      z = reinterpret_cast<const float*>(row.base)[token];
    else
      z = from_bf16(reinterpret_cast<const uint16_t*>(row.base)[token]);
    const double x = z == m ? 0.0 : ((double)z - (double)m) / (double)a.T;
    lp = (float)(x - log((double)total * p.unit));
  }
  p.logprob[r] = lp;
}

enum State : uint32_t { kDone = 0, kThreshold = 1, kRow = 2 };

template <int DT>
__global__ __launch_bounds__(kSegThreads) void sample_pick_kernel(SampleParams p) {
  __shared__ PickShared sh;
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  constexpr int NW = kSegThreads / 64;
  const int64_t r = blockIdx.x;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const Ask a = ask_of(p, r);
  const float* seg_max = p.seg_max + r * p.segs;
  const float m = row_max(seg_max, p.segs);
  if (t == 0 && p.state) p.state[r].what = kDone;
  if (!a.ok || !(m > kNegInf)) {  // NaN too
    if (t == 0) {
      p.token[r] = -1;
      if (p.logprob) p.logprob[r] = __builtin_nanf("");
    }
    return;
  }
  const R row = row_of<DT>(p, r);
  const Weights wt = weights_of(p, a, m);
  if (a.greedy || a.plain(p.V)) {
    // the segment that holds the token: the first with the maximum, or the one
    // in which the running sum crosses; every wavefront finds it
    u64 total = 0, before = 0;
    double goal = 0.0;
    if (!a.greedy) {
      for (int i = lane; i < p.segs; i += 64) total += p.seg_sum[r * p.segs + i];
      total = wave_sum(total);
      goal = (double)a.u * (double)total;
    }
    int seg = 0;
    for (int i = 0; i < p.segs; i += 64) {
      u64 v = 0;
      if (i + lane < p.segs)
        v = a.greedy ? (u64)(seg_max[i + lane] == m) : p.seg_sum[r * p.segs + i + lane];
      const u64 run = wave_scan(v);
      const uint64_t hit = __ballot(v != 0 && (double)(before + run) > goal);
      if (hit) {
        const int who = __builtin_ctzll(hit);
        seg = i + who;
        before += (u64)__shfl((unsigned long long)(run - v), who, 64);
        break;
      }
      before += (u64)__shfl((unsigned long long)run, 63, 64);
    }
    // 64 consecutive vectors are a chunk; its sum, then the chunk of the crossing
    auto amount = [&](float z) -> u64 { return a.greedy ? (u64)(z == m) : wt.all(z); };
    {
      float z[kVec][R::VE];
      load_group<DT>(row, seg * (kSegThreads * kVec) + t, z);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        u64 s = 0;
#pragma unroll
        for (int q = 0; q < R::VE; ++q) s += amount(z[j][q]);
        s = wave_sum(s);
        if (lane == 0) sh.hist[j * NW + wave] = s;
      }
    }
    __syncthreads();
    const u64 mine = lane < kVec * NW ? sh.hist[lane] : 0;
    const u64 run = wave_scan(mine);
    const uint64_t hit = __ballot(mine != 0 && (double)(before + run) > goal);
    const int chunk = hit ? __builtin_ctzll(hit) : 0;
    before += (u64)__shfl((unsigned long long)(run - mine), chunk, 64);
    if (wave == 0) {
      const int v = seg * (kSegThreads * kVec) + chunk * 64 + lane;
      u64 w[R::VE], s = 0;
#pragma unroll
      for (int q = 0; q < R::VE; ++q) w[q] = 0;
      if (v < row.nvec) {
        float z[R::VE];
        row.load(v, z);
#pragma unroll
        for (int q = 0; q < R::VE; ++q) {
          w[q] = amount(z[q]);
          s += w[q];
        }
      }
      const u64 upto = before + wave_scan(s);
      const uint64_t h = __ballot(s != 0 && (double)upto > goal);
      if (lane == (h ? __builtin_ctzll(h) : 0)) {
        u64 c = upto - s;
        int64_t token = -1;
#pragma unroll
        for (int q = 0; q < R::VE; ++q) {
          c += w[q];
          if (token < 0 && w[q] != 0 && (double)c > goal) token = row.first(v) + q;
        }
        write_out<DT>(p, r, row, a, m, token, total);
      }
    }
    return;
  }
  // candidates: distances up to hi
  float lo = 0.0f, hi = __builtin_huge_valf();
  u64 mass = 0, above = 0;
  bool threshold = false;
  if (a.list_all(p.V)) {
  } else if (a.hist(p.V)) {
    // the bin where the count or the mass is reached, 8 bins a thread
    constexpr int kPer = kBins / kSegThreads;
    const u64* hm = (const u64*)p.hist_mass + r * kBins + t * kPer;
    const uint32_t* hc = p.hist_count + r * kBins + t * kPer;
    u64 v = 0, c = 0;
    for (int j = 0; j < kPer; ++j) {
      c += hc[j];
      v += a.has_k ? (u64)hc[j] : hm[j];
    }
    if (!a.has_k) {
      for (int i = lane; i < p.segs; i += 64) mass += p.seg_sum[r * p.segs + i];
      mass = wave_sum(mass);
    }
    const double goal = a.has_k ? (double)a.k : a.p * (double)mass;
    const u64 rv = wave_scan(v), rc = wave_scan(c);
    if (lane == 63) {
      sh.wave[wave] = rv;
      sh.wave2[wave] = rc;
    }
    if (t == 0) {
      sh.out[0] = kBins - 1;  // never reached: all bins
      sh.out[1] = sh.out[2] = 0;
    }
    __syncthreads();
    u64 bv = rv - v, bc = rc - c;
    for (int i = 0; i < wave; ++i) {
      bv += sh.wave[i];
      bc += sh.wave2[i];
    }
    if (!reached(bv, goal, false) && reached(bv + v, goal, false)) {
      for (int j = 0; j < kPer; ++j) {
        const u64 w = a.has_k ? (u64)hc[j] : hm[j];
        bc += hc[j];
        if (reached(bv + w, goal, false)) {
          sh.out[0] = t * kPer + j;
          sh.out[1] = bv;
          sh.out[2] = bc;
          break;
        }
        bv += w;
      }
    }
    __syncthreads();
    const uint32_t bin = (uint32_t)sh.out[0];
    const uint32_t n_incl = (uint32_t)sh.out[2];
    // the distances of bin b lie between bits (base + b) << 16 and the next
    if (bin < kBins - 1) hi = __uint_as_float(((kBinBase + bin + 1) << 16) - 1);
    if (!a.has_k && n_incl > kCap) {
      threshold = true;
      above = sh.out[1];
      if (bin > 0) lo = __uint_as_float((kBinBase + bin) << 16);
    }
  } else if (a.has_k) {
    // k groups with maxima of at least the k-th largest hold k tokens as
    // large; the upper 16 bits of a key bound well enough
    const float* gm = p.group_max + r * p.segs * kSegThreads;
    const Sel s = radix_select(16, (double)a.k, false, sh, [&](auto f) {
      for (int g0 = 0; g0 < p.segs; g0 += kGroupBatch)
        each_group(gm, p.segs, g0, [&](int, float g) { f(Row<0>::key(g) >> 16, (u64)1); });
    });
    // fewer such groups than k: every token is a candidate
    if (s.above + s.at >= (u64)a.k) hi = distance(m, key_value<0>(s.key << 16));
  } else {
    // min-p alone: T ln(1 / min_p) and what its rounding may leave out
    hi = (float)(-(double)a.T * log(a.minp) * (1.0 + 1e-6)) + 1e-30f;
    hi += hi * 1e-6f;
  }
  const uint32_t n = gather_groups<DT>(row, p, r, wt, lo, hi, sh);
  if (n > kCap) {
    // min-p alone keeps all it has gathered: no further threshold
    if (t == 0) {
      p.state[r].what = !a.has_k && !a.has_p ? kThreshold : kRow;
      p.state[r].tau = 0;
      p.state[r].ties = 0;
    }
    return;
  }
  if (a.list_all(p.V) && a.has_p && !a.has_k) {
    u64 v = 0;
    for (uint32_t i = t; i < n; i += kSegThreads) v += sh.list[i].q & ~kKeptBit;
    mass = block_sum<NW>(v, sh);
  }
  const Drawn d = draw_list<DT>(a, wt, p.V, n, mass, threshold, above, sh);
  if (t == 0) {
    if (threshold) {
      p.state[r].what = kThreshold;
      p.state[r].tau = d.tau;
      p.state[r].ties = d.ties;
    } else {
      write_out<DT>(p, r, row, a, m, d.token, d.total);
    }
  }
}

// Rows with a threshold and no token yet: a segment's kept weight above the
// threshold's key, and its tokens of that key.
template <int DT>
__global__ __launch_bounds__(kSegThreads, 4) void sample_kept_kernel(SampleParams p) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  __shared__ u64 part[2][kSegThreads / 64];
  const int64_t r = blockIdx.x;
  if (p.state[r].what != kThreshold) return;
  const int seg = blockIdx.y, t = threadIdx.x;
  const Ask a = ask_of(p, r);
  const float m = row_max(p.seg_max + r * p.segs, p.segs);
  const Weights wt = weights_of(p, a, m);
  const R row = row_of<DT>(p, r);
  const uint32_t tau = p.state[r].tau;
  float z[kVec][R::VE];
  load_group<DT>(row, seg * (kSegThreads * kVec) + t, z);
  u64 s = 0, c = 0;
#pragma unroll
  for (int j = 0; j < kGroup; ++j) {
    const float v = z[j / R::VE][j % R::VE];
    const uint32_t k = R::key(v);
    if (k > tau) s += wt.kept(v);
    c += k == tau && v != kNegInf;
  }
  s = wave_sum(s);
  c = wave_sum(c);
  if ((t & 63) == 0) {
    part[0][t >> 6] = s;
    part[1][t >> 6] = c;
  }
  __syncthreads();
  if (t == 0) {
    p.seg_sum[r * p.segs + seg] = part[0][0] + part[0][1] + part[0][2] + part[0][3];
    p.seg_ties[r * p.segs + seg] =
        (uint32_t)(part[1][0] + part[1][1] + part[1][2] + part[1][3]);
  }
}

// Draws where the candidates do not fit in LDS: every pass reads the row.
template <int DT>
__device__ __forceinline__ Drawn draw_row(const Row<DT>& row, const Ask& a, const Weights& wt, Shared& sh) {
  typedef Row<DT> R;
  const float m = wt.m;
  bool has_k = a.has_k;
  uint32_t tau = 0;
  int64_t last = row.V;
  bool select = false;  // tau is set
  u64 ties = 0;
  uint32_t n_list = 0;
  // f(z, index) over the list, or over the row's tokens of bin b
  auto over = [&](bool list, uint32_t b, auto f) {
    if (list) {
      for (uint32_t i = threadIdx.x; i < n_list; i += kThreads)
        f(__uint_as_float(sh.key[i]), (int64_t)sh.idx[i]);
    } else {
      row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t e, const float* z) {
#pragma unroll
        for (int j = 0; j < R::VE; ++j) {
          if (z[j] == kNegInf) continue;
          if (bin_of(m, z[j]) == b) f(z[j], e + j);
        }
      });
    }
  };
  u64 mass_k = 0;
  if (has_k) {
    histogram<DT, false>(row, wt, sh);
    const BinSel b = scan_bins(sh, [&](int i) { return (u64)sh.count[i]; },
                               [&](u64) { return (double)a.k; });
    if (b.total <= (u64)a.k) {
      has_k = false;  // fewer admissible tokens than k
    } else {
      select = true;
      const bool list = b.n_at <= kCap;
      if (list) {
        gather<DT>(row, wt, sh, b.bin, b.bin);
        n_list = min(sh.n, (uint32_t)kCap);
      }
      const Sel s = radix_select(R::kKeyBits, (double)((u64)a.k - b.above), false, sh,
                                 [&](auto f) {
        over(list, b.bin, [&](float z, int64_t) { f(R::key(z), (u64)1); });
      });
      tau = s.key;
      ties = (u64)a.k - b.above - s.above;
      if (a.has_p) {
        u64 v = 0;
        row.each(0, row.nvec, threadIdx.x, kThreads, [&](int64_t, const float* z) {
#pragma unroll
          for (int j = 0; j < R::VE; ++j)
            if (R::key(z[j]) > tau) v += wt.all(z[j]);
        });
        mass_k = block_sum<kWaves>(v, sh) + ties * wt.all(key_value<DT>(tau));
      }
    }
  }
  if (a.has_p) {
    histogram<DT, true>(row, wt, sh);
    const BinSel b = scan_bins(sh, [&](int i) { return sh.mass[i]; }, [&](u64 total) {
      return a.p * (double)(has_k ? mass_k : total);
    });
    const double goal = a.p * (double)(has_k ? mass_k : b.total);
    const bool list = b.n_at <= kCap;
    if (list) {
      gather<DT>(row, wt, sh, b.bin, b.bin);
      n_list = min(sh.n, (uint32_t)kCap);
    }
    const uint32_t tau_k = tau;
    const Sel s = radix_select(R::kKeyBits, goal - (double)b.above, false, sh, [&](auto f) {
      over(list, b.bin, [&](float z, int64_t) {
        if (R::key(z) >= tau_k) f(R::key(z), wt.all(z));
      });
    });
    u64 n = 0;
    over(list, b.bin, [&](float z, int64_t) { n += R::key(z) == s.key; });
    n = block_sum<kWaves>(n, sh);
    if (select && s.key == tau_k && ties < n) n = ties;
    ties = ties_needed(b.above + s.above, wt.all(key_value<DT>(s.key)), n, goal);
    tau = s.key;
    select = true;
  }
  if (select) {
    u64 n;
    last = locate<DT>(row, 0, row.nvec, sh, 0, [&](u64) { return (double)ties - 0.5; }, &n,
                      [&](int64_t, float z) {
      return (u64)(z != kNegInf && R::key(z) == tau);
    });
  }
  Drawn d;
  d.token = locate<DT>(row, 0, row.nvec, sh, 0,
                       [&](u64 all) { return (double)a.u * (double)all; }, &d.total,
                       [&](int64_t i, float z) -> u64 {
    if (!select) return wt.kept(z);
    const uint32_t k = R::key(z);
    return k > tau || (k == tau && i <= last) ? wt.kept(z) : 0;
  });
  return d;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_rest_kernel(SampleParams p) {
  __shared__ Shared sh;
  typedef Row<DT> R;
  const int64_t r = blockIdx.x;
  const uint32_t what = p.state[r].what;
  if (what == kDone) return;
  const Ask a = ask_of(p, r);
  const float m = row_max(p.seg_max + r * p.segs, p.segs);
  const R row = row_of<DT>(p, r);
  const Weights wt = weights_of(p, a, m);
  Drawn d;
  if (what == kRow) {
    d = draw_row<DT>(row, a, wt, sh);
  } else {
    // the segment in which the kept sum crosses; the ties kept are the first
    // in index order, so a segment has those that the ones before it left
    const int lane = threadIdx.x & 63;
    const uint32_t tau = p.state[r].tau;
    const u64 ties = p.state[r].ties;
    const u64 each = ties ? wt.kept(key_value<DT>(tau)) : 0;
    const u64* sum = (const u64*)p.seg_sum + r * p.segs;
    const uint32_t* cnt = p.seg_ties + r * p.segs;
    u64 total = 0;
    for (int i = lane; i < p.segs; i += 64) total += sum[i];
    total = wave_sum(total) + ties * each;
    const double goal = (double)a.u * (double)total;
    u64 before = 0, used = 0, here = 0, all_here = 0;
    int seg = 0;
    for (int i = 0; i < p.segs; i += 64) {
      const bool in = i + lane < p.segs;
      const u64 c = in ? cnt[i + lane] : 0;
      const u64 c_before = used + wave_scan(c) - c;
      const u64 left = ties > c_before ? ties - c_before : 0;
      const u64 k = left < c ? left : c;
      const u64 v = (in ? sum[i + lane] : 0) + k * each;
      const u64 run = wave_scan(v);
      const uint64_t hit = __ballot(v != 0 && (double)(before + run) > goal);
      if (hit) {
        const int who = __builtin_ctzll(hit);
        seg = i + who;
        before += (u64)__shfl((unsigned long long)(run - v), who, 64);
        here = (u64)__shfl((unsigned long long)k, who, 64);
        all_here = (u64)__shfl((unsigned long long)c, who, 64);
        break;
      }
      before += (u64)__shfl((unsigned long long)run, 63, 64);
      used = (u64)__shfl((unsigned long long)(c_before + c), 63, 64);
    }
    constexpr int kSegVec = kSeg / R::VE;
    const int c0 = seg * kSegVec, c1 = min(c0 + kSegVec, row.nvec);
    int64_t last = here == all_here ? row.V : -1;
    u64 part;
    if (here != 0 && here < all_here)
      last = locate<DT>(row, c0, c1, sh, 0, [&](u64) { return (double)here - 0.5; }, &part,
                        [&](int64_t, float z) {
        return (u64)(z != kNegInf && R::key(z) == tau);
      });
    d.total = total;
    d.token = locate<DT>(row, c0, c1, sh, before, [&](u64) { return goal; }, &part,
                         [&](int64_t i, float z) -> u64 {
      const uint32_t k = R::key(z);
      return k > tau || (k == tau && i <= last) ? wt.kept(z) : 0;
    });
  }
  if (threadIdx.x == 0) write_out<DT>(p, r, row, a, m, d.token, d.total);
}

}  // namespace

// Bits after the point of a weight: the sum over V of them stays below 2^63.
static int weight_bits(int64_t V) {
  int n = 0;
  while (((int64_t)1 << n) < V) ++n;
  const int fb = 62 - n;
  return fb < 44 ? fb : 44;
}

static int64_t segments(int64_t V) { return (V + 8 + kSeg - 1) / kSeg; }

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

size_t sample_workspace_bytes(int64_t N, int64_t V) {
  const size_t rows = (size_t)N, s = rows * (size_t)segments(V);
  return 256 + up256(s * kSegThreads * 4) + 2 * up256(s * 4) + up256(s * 8) +
         up256(rows * kBins * 8) + up256(rows * kBins * 4) + up256(rows * sizeof(SampleState));
}

hipError_t launch_sample(SampleParams p, int dtype, int64_t N, void* workspace,
                         hipStream_t stream) {
  if (N <= 0) return hipSuccess;
  // (2^f - 1) / f on [-1/2, 1/2], from the constant term up (see Weights)
  static const double kPoly[9] = {0x1.62e42fefa39efp-1,  0x1.ebfbdff823cedp-3,
                                  0x1.c6b08d7047e52p-5,  0x1.3b2ab7181b755p-7,
                                  0x1.5d87fe86fe88ep-10, 0x1.4308ac85aa947p-13,
                                  0x1.ffcb9515a8016p-17, 0x1.63d136366db24p-20,
                                  0x1.b63880a30e9ffp-24};
  for (int i = 0; i < 9; ++i) p.poly[i] = kPoly[i];
  const int fb = weight_bits(p.V);
  p.magic = ldexp(1.0, 52 - fb);
  p.unit = ldexp(1.0, -fb);
  p.segs = (int)segments(p.V);
  const size_t rows = (size_t)N, s = rows * (size_t)p.segs;
  char* w = static_cast<char*>(workspace);
  auto take = [&](size_t n) {
    char* at = w;
    w += up256(n);
    return at;
  };
  p.group_max = reinterpret_cast<float*>(take(s * kSegThreads * 4));
  p.seg_max = reinterpret_cast<float*>(take(s * 4));
  p.seg_ties = reinterpret_cast<uint32_t*>(take(s * 4));
  p.seg_sum = reinterpret_cast<unsigned long long*>(take(s * 8));
  p.hist_mass = reinterpret_cast<unsigned long long*>(take(rows * kBins * 8));
  p.hist_count = reinterpret_cast<uint32_t*>(take(rows * kBins * 4));
  p.state = reinterpret_cast<SampleState*>(take(rows * sizeof(SampleState)));
  const dim3 seg_grid((unsigned)N, (unsigned)p.segs);
  // rows of at most kCap tokens are gathered whole; without filters no row has
  // more candidates than LDS holds
  const bool mass = p.V > kCap;
  const bool rest = mass && (p.top_k || p.top_p || p.min_p);
  if (!rest) p.state = nullptr;
  auto run = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    hipLaunchKernelGGL((sample_max_kernel<DT>), seg_grid, dim3(kSegThreads), 0, stream, p);
    if (mass)
      hipLaunchKernelGGL((sample_mass_kernel<DT>), seg_grid, dim3(kSegThreads), 0, stream, p);
    hipLaunchKernelGGL((sample_pick_kernel<DT>), dim3((unsigned)N), dim3(kSegThreads), 0, stream,
                       p);
    if (rest) {
      hipLaunchKernelGGL((sample_kept_kernel<DT>), seg_grid, dim3(kSegThreads), 0, stream, p);
      hipLaunchKernelGGL((sample_rest_kernel<DT>), dim3((unsigned)N), dim3(kThreads), 0, stream,
                         p);
    }
  };
  if (dtype == 0)
    run(std::integral_constant<int, 0>{});
  else
    run(std::integral_constant<int, 1>{});
  return hipGetLastError();
}

}  // namespace vce
