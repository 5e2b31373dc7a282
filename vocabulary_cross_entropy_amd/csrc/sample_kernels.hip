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
//    the segment's weights for rows without filters, and for rows whose top-p stands
//    alone (or whose top-k is large) adds the segment to the row's
//    histogram over the distance m - z (128 bins per octave, 16 octaves).
//  * sample_pick_kernel (rows) draws.  Candidates are bounded from below first: by
//    the k-th largest group maximum (k groups hold at least k tokens as
//    large), by the histogram's bin where the mass or the count is reached, or by min-p
//    itself; only groups that reach the bound are read again and their
//    candidates gathered in LDS.  Up to 64 are ranked by counting, more go
//    through selection by nine key bits at a time.  A row without filters
//    re-reads the one segment in which its sum crosses u.  Rows of up to 4096 tokens
//    make their own histogram here and need none of the other kernels but the first.
//  * rows with more candidates than LDS holds: sample_kept_kernel (rows x
//    segments) sums what lies before the histogram's bin and lists the tokens of
//    that bin, sample_rest_kernel (rows) finds the threshold in the list and
//    draws.  (For few segments each of these pairs, mass and pick, kept and rest, is
//    one launch; the last workgroup of a row goes on with the row.)  What does not fit that either (a large top-k together with top-p, more ties
//    than the list holds) is served from the row, pass by pass: 16 x 200000 with top-k
//    20000 and top-p 0.99 take 370 us against 43 for a top-k of 5000.
//
// What bounds it: sample_max_kernel memory (256 x 128256 BF16 14 us, 4.8 TB/s), the
// weights of a segment FP64 issue (22 instructions a token: 61 x 256003 FP32 without
// filters 21 us), and sample_pick_kernel and sample_rest_kernel, one workgroup a row,
// the latency of some dozen steps between barriers (256 rows of top-k 50 18 us, of
// top-k 1000 29 us).  256 x 128256 BF16 of mixed parameters take 95 us (max 14, mass
// 21, pick 32, kept 10, rest 20), one row with all filters 18 to 21 us.  512 threads a
// row: with 256 the mixed rows took 118 us where 512 took 110, with 1024 no less.  The code
// that a usual row runs is kept short, too: a kernel this brief waits for its instructions
// as well as for its data.
//
#include <math.h>

#include <type_traits>

#include "vce_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

constexpr int kThreads = 256;  // of a segment's workgroup
constexpr int kWaves = kThreads / 64;
constexpr int kRowThreads = 512;  // of a row's
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kBins = 2048;
constexpr uint32_t kBinBase = 119u << 7;  // bits of 2^-8 over 2^16: bin 0 lies below
constexpr int kCap = 4096;                // candidates held in LDS
// Ranked by counting, every one against every other, by one wavefront.  With 256, 256 rows
// of top-k 200 took 38 us against 21 by selection, top-k 50 17 us either way.
constexpr int kRank = 64;
constexpr int kLoads = 4;                 // vectors in flight per thread
constexpr int kGroup = 32;                // tokens per thread of a segment
constexpr int kSeg = kThreads * kGroup;
// Row segments up to which a segments' and a rows' kernel are one launch: a workgroup per
// CU.  Below, a launch less saves 1 to 4 us (one row of 128256 with all filters 23.6 ->
// 21.0 us); with more, the segments run at the rows' kernels' two workgroups per CU
// (1024 segments of top-p 70 -> 96 us).
constexpr int kJoined = 256;
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
  // The same in two parts, so that several vectors' loads wait together: the load
  // where the row fills the vector, then its logits, -inf for a vector past the row.
  __device__ __forceinline__ bool full(int i) const {
    const int64_t e = first(i);
    return e >= 0 && e + VE <= V;
  }
  __device__ __forceinline__ u32x4_t raw(int i) const {
    return *reinterpret_cast<const u32x4_t*>(base + first(i) * (DT == 0 ? 4 : 2));
  }
  __device__ __forceinline__ void take(int i, const u32x4_t& w, float* z) const {
    if (full(i)) {
      unpack(w, z);
    } else if (i < nvec) {
      load(i, z);
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) z[j] = kNegInf;
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
  // x below -64 rounds to no weight.  real() is for a finite m.
  __device__ __forceinline__ double real(float z) const { return power((double)z - md); }
  // The same whatever m is: where it is infinite z = m has weight 1, all else
  // none.  No branch, so that many run interleaved.
  __device__ __forceinline__ double weight(float z) const {
    return power(z == m ? 0.0 : (double)z - md);
  }
  __device__ __forceinline__ double power(double d) const {
    double x = d * c;
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

constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;  // of a radix selection

constexpr int kGroupBatch = 8;   // group maxima that a thread loads at once
constexpr int kKeepSegs = 1024;  // segments of a row that sample_rest_kernel draws from

struct Scratch {
  union {
    u64 hist[3 * kDigits];
    uint16_t group[kGroupBatch * kRowThreads];
    u64 keep[kKeepSegs];
  };
  u64 wave[kRowWaves];
  u64 wave2[kRowWaves];
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

struct PickShared : Scratch {
  Entry list[kCap];
  uint32_t n_groups;
};

// v of another lane of the wavefront by data-parallel-primitive control CTRL, 0
// where there is none.
template <int CTRL, int ROWS>
__device__ __forceinline__ u64 dpp64(u64 v) {
  const int lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)v, CTRL, ROWS, 0xf, false);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(v >> 32), CTRL, ROWS, 0xf, false);
  return ((u64)(uint32_t)hi << 32) | (uint32_t)lo;
}

// Running sum over the lanes, each with its own share included: within rows of
// 16 lanes by shifts, then row 0 into row 1 and 2 into 3, then lane 31 into the
// upper half.  (Register moves; a shuffle through LDS per step took ten times as long.)
__device__ __forceinline__ u64 wave_scan(u64 v) {
  v += dpp64<0x111, 0xf>(v);
  v += dpp64<0x112, 0xf>(v);
  v += dpp64<0x114, 0xf>(v);
  v += dpp64<0x118, 0xf>(v);
  v += dpp64<0x142, 0xa>(v);
  v += dpp64<0x143, 0xc>(v);
  return v;
}

__device__ __forceinline__ u64 lane64(u64 v, int lane) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane);
  return ((u64)hi << 32) | lo;
}

__device__ __forceinline__ u64 wave_sum(u64 v) { return lane64(wave_scan(v), 63); }

// Sum over the workgroup, the same in every thread.
template <class S>
__device__ __forceinline__ u64 block_sum(u64 v, S& sh) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh.wave[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kRowWaves; ++i) v += sh.wave[i];
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
// Every wavefront scans the digit's histogram for itself, and three histograms
// take turns: one barrier per digit.
template <class S, class Visit>
__device__ __forceinline__ Sel radix_select(int bits, double target, bool strict, S& sh,
                                            Visit visit) {
  constexpr int kPer = kDigits / 64;
  const int lane = threadIdx.x & 63;
  uint32_t prefix = 0;
  u64 above = 0, at = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < kDigits; i += kRowThreads) sh.hist[i] = 0;
  __syncthreads();
  int buf = 0;
  for (int shift = (bits - 1) / kDigitBits * kDigitBits; shift >= 0; shift -= kDigitBits) {
    u64* hist = sh.hist + buf * kDigits;
    visit([&](uint32_t k, u64 a) {
      if (a != 0 && (k >> shift >> kDigitBits) == prefix)
        atomicAdd(&hist[(k >> shift) & (kDigits - 1)], a);
    });
    // the next digit's, which was scanned two digits ago: every wavefront has
    // passed the barrier since
    buf = buf == 2 ? 0 : buf + 1;
    u64* clear = sh.hist + buf * kDigits;
    for (int i = threadIdx.x; i < kDigits; i += kRowThreads) clear[i] = 0;
    __syncthreads();
    u64 h[kPer], s = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      h[j] = hist[kDigits - 1 - kPer * lane - j];
      s += h[j];
    }
    const u64 run = wave_scan(s);
    const uint64_t hit = __ballot(reached(above + run, target, strict));
    const uint64_t some = __ballot(s != 0);
    // the first lane that reaches it, else the last that holds anything
    const int who = hit ? __builtin_ctzll(hit) : some ? 63 - __builtin_clzll(some) : 63;
    // in that lane: the first of its digits that reaches it, else its last that
    // holds anything
    u64 a = above + run - s, pick_above = a, pick_at = 0;
    int pick = 0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (!found && h[j] != 0) {
        pick = j;
        pick_above = a;
        pick_at = h[j];
        found = reached(a + h[j], target, strict);
      }
      a += h[j];
    }
    prefix = (prefix << kDigitBits) |
             (uint32_t)(kDigits - 1 - kPer * who -
                        __builtin_amdgcn_readlane(pick, who));
    above = lane64(pick_above, who);
    at = lane64(pick_at, who);
  }
  return Sel{prefix, above, at};
}

// The first index, in order, of vectors [c0, c1) at which the running sum of
// amount(index, z), from `before` on, exceeds target(sum of the range); V if it
// never does.  Each wavefront sums a
// share of the range, the share that holds the crossing is split
// again, down to one vector per lane.
template <int DT, class Target, class Amount>
__device__ __forceinline__ int64_t locate(const Row<DT>& row, int c0, int c1, Shared& sh, u64 before,
                          Target target, u64* total, Amount amount) {
  constexpr int VE = Row<DT>::VE;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double goal = 0.0;
  bool first = true;
  while (true) {
    const int chunk = (c1 - c0 + kRowWaves - 1) / kRowWaves;
    const int a = min(c0 + wave * chunk, c1), b = min(a + chunk, c1);
    u64 s = 0;
    row.each(a, b, lane, 64, [&](int64_t e, const float* z) {
#pragma unroll
      for (int j = 0; j < VE; ++j) s += amount(e + j, z[j]);
    });
    s = wave_sum(s);
    __syncthreads();
    if (lane == 0) sh.wave[wave] = s;
    __syncthreads();
    if (first) {
      u64 all = 0;
#pragma unroll
      for (int i = 0; i < kRowWaves; ++i) all += sh.wave[i];
      *total = all;
      goal = target(all);
      first = false;
    }
    int w = -1;
    for (int i = 0; i < kRowWaves; ++i) {
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
    const u64 run = wave_scan(s);
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
  for (int i = threadIdx.x; i < kBins; i += kRowThreads) {
    sh.count[i] = 0;
    sh.mass[i] = 0;
  }
  __syncthreads();
  row.each(0, row.nvec, threadIdx.x, kRowThreads, [&](int64_t, const float* z) {
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
  constexpr int kPer = kBins / kRowThreads;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  u64 s = 0;
  uint32_t n = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    s += amount(t * kPer + j);
    n += sh.count[t * kPer + j];
  }
  const u64 run = wave_scan(s), cnt = wave_scan(n);
  __syncthreads();
  if (lane == 63) {
    sh.wave[wave] = run;
    sh.wave2[wave] = cnt;
  }
  __syncthreads();
  u64 base = 0, nbase = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kRowWaves; ++i) {
    if (i < wave) {
      base += sh.wave[i];
      nbase += sh.wave2[i];
    }
    total += sh.wave[i];
  }
  const double goal = target(total);
  // exactly one thread's bins hold the crossing: before it not reached, with it reached
  const u64 before = base + run - s, upto = base + run;
  if (t == kRowThreads - 1) {
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
  row.each(0, row.nvec, threadIdx.x, kRowThreads, [&](int64_t e, const float* z) {
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
  // so short a row that LDS holds all of it: sample_pick_kernel alone serves it
  __device__ __forceinline__ bool small(int64_t V) const { return V <= kCap; }
  // few enough tokens asked for that the group maxima bound them closely
  __device__ __forceinline__ bool group_bound(int64_t V) const {
    return has_k && k <= kSmallK && k <= V / (4 * kGroup);
  }
  // by the histogram: top-p alone, or a top-k too large for the group maxima
  __device__ __forceinline__ bool hist(int64_t V) const {
    return ok && !greedy && !small(V) && (has_k ? !group_bound(V) : has_p);
  }
  __device__ __forceinline__ bool plain() const {
    return ok && !greedy && !has_k && !has_p && !has_min;
  }
};

// The launcher points an absent parameter at u: the loads have no branch
// between them and wait together.
__device__ __forceinline__ Ask ask_of(const SampleParams& p, int64_t r) {
  Ask a;
  const float T = p.temperature[r], top_p = p.top_p[r], min_p = p.min_p[r];
  const int32_t k = p.top_k[r];
  a.u = p.u[r];
  a.T = p.has & SampleParams::kT ? T : 1.0f;
  const float pp = p.has & SampleParams::kP ? top_p : 1.0f;
  const float mp = p.has & SampleParams::kM ? min_p : 0.0f;
  a.k = p.has & SampleParams::kK ? k : 0;
  // written so that a NaN fails
  a.ok = a.T >= 0.0f && a.T < __builtin_huge_valf() && a.u >= 0.0f && a.u < 1.0f && pp == pp &&
         mp == mp;
  a.greedy = a.T == 0.0f;
  a.has_k = a.k > 0 && a.k < p.V;
  a.has_p = pp < 1.0f;
  a.has_min = mp > 0.0f;
  a.p = fmaxf(pp, 0.0f);      // the first token is always kept
  a.minp = fminf(mp, 1.0f);   // and so are the maxima
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
  // below 2^22 rows
  const uint32_t i0 = (uint32_t)r / (uint32_t)p.d1, i1 = (uint32_t)r - i0 * (uint32_t)p.d1;
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

// The tokens of a thread of a segment that NT threads share: vectors v0, v0 + NT,
// ... of the row, -inf past its ends.  The loads are issued by load() and waited
// for by get().
template <int DT, int NT>
struct Group {
  typedef Row<DT> R;
  static constexpr int kVec = kSeg / NT / R::VE;
  u32x4_t raw[kVec];
  bool full;
  __device__ __forceinline__ void load(const R& row, int v0) {
    const int last = v0 + (kVec - 1) * NT;
    full = last < (int)((row.V + row.off) / R::VE) && (v0 > 0 || row.off == 0);
    if (full) {
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        raw[j] = *reinterpret_cast<const u32x4_t*>(row.base + row.first(v0 + j * NT) *
                                                                  (DT == 0 ? 4 : 2));
    }
  }
  __device__ __forceinline__ void get(const R& row, int v0, float (&z)[kVec][R::VE]) const {
    if (full) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) R::unpack(raw[j], z[j]);
    } else {
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (v0 + j * NT < row.nvec) {
          row.load(v0 + j * NT, z[j]);
        } else {
#pragma unroll
          for (int q = 0; q < R::VE; ++q) z[j][q] = kNegInf;
        }
      }
    }
  }
};

// The workgroup's row and segment.  Segments run fastest: workgroups are dealt
// round-robin over the XCDs, and rows differ in what they ask for, so each row's
// segments go to all of them (with rows running fastest 256 mixed rows left some XCDs
// with half as much again to do).
__device__ __forceinline__ bool row_and_segment(const SampleParams& p, int64_t* r, int* seg) {
  const uint32_t b = blockIdx.y * gridDim.x + blockIdx.x;
  const uint32_t row = b / (uint32_t)p.segs;
  *r = row;
  *seg = (int)(b - row * (uint32_t)p.segs);
  return row < p.rows;
}

template <int DT>
__global__ __launch_bounds__(kThreads) void sample_max_kernel(SampleParams p) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  __shared__ float sh[kThreads / 64];
  int64_t r;
  int seg;
  if (!row_and_segment(p, &r, &seg)) return;
  const int t = threadIdx.x;
  const R row = row_of<DT>(p, r);
  float z[kVec][R::VE];
  Group<DT, kThreads> group;
  group.load(row, seg * (kThreads * kVec) + t);
  group.get(row, seg * (kThreads * kVec) + t, z);
  float m = kNegInf;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kVec; ++j)
#pragma unroll
    for (int q = 0; q < R::VE; ++q) {
      m = fmaxf(m, z[j][q]);
      nan |= z[j][q] != z[j][q];
    }
  p.group_max[(r * p.segs + seg) * kThreads + t] = m;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  if (__any(nan)) m = __builtin_nanf("");
  if ((t & 63) == 0) sh[t >> 6] = m;
  if (seg == 0 && t < 2 && p.done) p.done[2 * r + t] = 0;
  // the row's histogram starts at zero, a share of it per segment
  if (ask_of(p, r).hist(p.V)) {
    for (int64_t b = seg * kThreads + t; b < kBins; b += (int64_t)p.segs * kThreads)
      p.hist[r * kBins + b] = 0;
  }
  __syncthreads();
  if (t == 0) {
    bool any = false;
    float s = kNegInf;
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) {
      any |= sh[i] != sh[i];
      s = fmaxf(s, sh[i]);
    }
    p.seg_max[r * p.segs + seg] = any ? __builtin_nanf("") : s;
  }
}

// Words that the workgroups of a row hand to the last of them within a launch go past the
// caches of the XCDs, by device-scope atomic stores and loads.
template <class T>
__device__ __forceinline__ void put_shared(T* at, T v) {
  __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class T>
__device__ __forceinline__ T get_shared(const T* at) {
  return __hip_atomic_load(const_cast<T*>(at), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// True in the last of a row's workgroups to come here.  Every wavefront first waits
// until its device-scope stores and atomics are done; then the workgroup is counted.  (A
// release fence at device scope writes a whole L2 back: with one per workgroup 256 mixed
// rows took 521 us.)
__device__ __forceinline__ bool last_of_row(uint32_t* count, int segs, Scratch& sh) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) sh.n = atomicAdd(count, 1u);
  __syncthreads();
  const bool last = sh.n == (uint32_t)segs - 1;
  __syncthreads();
  return last;
}

// For rows without filters the segment's mass; for rows that go by the
// histogram its tokens per bin (top-k), or its mass per bin and in all (top-p).
// Top-p needs no token lighter than q0 = (1 - p) / V: the row's mass is at least
// 1, so all such tokens together weigh less than (1 - p) of it, and its p-th part is
// reached before them.  They stay out of the histogram, which spares most of the
// LDS atomics.
template <int DT, int NT>
__device__ __forceinline__ void mass_of_segment(const SampleParams& p, const Row<DT>& row,
                                                const Ask& a, int64_t r, int seg, u64* bins,
                                                u64* part) {
  typedef Row<DT> R;
  typedef Group<DT, NT> G;
  constexpr int kVec = G::kVec, kTokens = kVec * R::VE;
  const bool plain = a.plain(), hist = !plain;
  const int t = threadIdx.x;
  const int v0 = seg * (kSeg / R::VE) + t;
  G group;
  group.load(row, v0);
  const float m = row_max(p.seg_max + r * p.segs, p.segs);
  if (!(m > kNegInf)) return;  // no admissible token, or NaN
  const Weights wt = weights_of(p, a, m);
  u64 s = 0, q0 = 0;
  if (hist) {
    for (int b = t; b < kBins; b += NT) bins[b] = 0;
    q0 = wt.fixed((1.0 - a.p) * p.inv_v);
    q0 = q0 < 1 ? 1 : q0;
    __syncthreads();
  }
  float z[kVec][R::VE];
  group.get(row, v0, z);
  if (plain && !wt.inf) {
    // eight at a time: enough to fill the pipeline
#pragma unroll
    for (int j0 = 0; j0 < kTokens; j0 += 8) {
#pragma unroll
      for (int j = j0; j < j0 + 8; ++j) s += wt.fixed(wt.real(z[j / R::VE][j % R::VE]));
      __builtin_amdgcn_sched_barrier(0);
    }
  } else if (hist && a.has_k) {
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      const float v = z[j / R::VE][j % R::VE];
      if (v != kNegInf) atomicAdd(&bins[bin_of(m, v)], (u64)1);
    }
  } else if (!wt.inf) {
    // eight weights at a time, interleaved, then their atomics
#pragma unroll
    for (int j0 = 0; j0 < kTokens; j0 += 8) {
      u64 q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[j] = wt.fixed(wt.real(z[(j0 + j) / R::VE][(j0 + j) % R::VE]));
        s += q[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (q[j] >= q0) atomicAdd(&bins[bin_of(m, z[(j0 + j) / R::VE][(j0 + j) % R::VE])], q[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
    // only the infinite tokens weigh, all in bin 0
#pragma unroll
    for (int j = 0; j < kTokens; ++j) s += wt.all(z[j / R::VE][j % R::VE]);
    if (hist && s) atomicAdd(&bins[0], s);
  }
  s = wave_sum(s);
  if ((t & 63) == 0) part[t >> 6] = s;
  __syncthreads();
  if (t == 0) {
    s = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) s += part[i];
    put_shared(&p.seg_sum[r * p.segs + seg], s);
  }
  if (hist) {
    for (int b = t; b < kBins; b += NT)
      if (bins[b]) atomicAdd((u64*)&p.hist[r * kBins + b], bins[b]);
  }
}

// What sample_mass_kernel has to do for a row.
__device__ __forceinline__ bool needs_mass(const Ask& a, int64_t V) {
  return a.hist(V) || (a.plain() && !a.small(V));
}

template <int DT>
__global__ __launch_bounds__(kThreads, 4) void sample_mass_kernel(SampleParams p) {
  __shared__ u64 bins[kBins];
  __shared__ u64 part[kWaves];
  int64_t r;
  int seg;
  if (!row_and_segment(p, &r, &seg)) return;
  const Ask a = ask_of(p, r);
  if (!needs_mass(a, p.V)) return;
  mass_of_segment<DT, kThreads>(p, row_of<DT>(p, r), a, r, seg, bins, part);
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

template <int DT>
__device__ __forceinline__ Entry entry_of(const Weights& wt, float z, uint32_t idx) {
  const double w = wt.weight(z);
  return Entry{Row<DT>::key(z), idx, wt.fixed(w) | (w >= wt.minp ? kKeptBit : 0)};
}

// m - z, 0 for z = m also where both are infinite.
__device__ __forceinline__ float distance(float m, float z) { return z == m ? 0.0f : m - z; }

// The maxima of the row's groups, kGroupBatch per thread at a time with their
// loads in flight together; the first ones stay in registers.
struct GroupMax {
  static constexpr int kBatch = kGroupBatch * kRowThreads;
  const float* gm;  // (segs, 256) of the row
  int n;
  float first[kGroupBatch];
  __device__ __forceinline__ void load(int g0, float (&top)[kGroupBatch]) const {
#pragma unroll
    for (int i = 0; i < kGroupBatch; ++i) {
      const int g = g0 + i * kRowThreads + (int)threadIdx.x;
      top[i] = g < n ? gm[g] : kNegInf;
    }
  }
  __device__ __forceinline__ void init(const float* p, int segs) {
    gm = p;
    n = segs * kThreads;
    load(0, first);
  }
  // f(group, maximum) for the groups g0 .. g0 + kBatch - 1, counted from g0.
  template <class F>
  __device__ __forceinline__ void each(int g0, F f) const {
    float top[kGroupBatch];
#pragma unroll
    for (int i = 0; i < kGroupBatch; ++i) top[i] = first[i];
    if (g0) load(g0, top);
#pragma unroll
    for (int i = 0; i < kGroupBatch; ++i)
      if (top[i] != kNegInf) f(i * kRowThreads + (int)threadIdx.x, top[i]);
  }
};

// Gathers into LDS the tokens with m - z <= hi, in no order, from the groups
// whose maximum is within it: first those groups are listed, then their vectors
// are dealt over the threads, so that the loads wait together.  Returns the
// number of tokens; the list is not whole where that is above kCap, or where
// more than max_groups groups are listed (the number returned is then above
// kCap as well).
template <int DT>
__device__ __forceinline__ uint32_t gather_groups(const Row<DT>& row, const GroupMax& groups,
                                                  const Weights& wt, float hi,
                                                  uint32_t max_groups, PickShared& sh) {
  typedef Row<DT> R;
  constexpr int kVec = kGroup / R::VE;
  constexpr int kItems = 2;  // vectors in flight per thread
  __syncthreads();
  if (threadIdx.x == 0) sh.n = 0;
  // sh.n as every batch of groups starts.  It decides whether the batch still fits, and comes from
  // a register: wavefronts that are already gathering the batch add to sh.n, and one that read it
  // late could leave alone.
  uint32_t have = 0;
  for (int g0 = 0; g0 < groups.n; g0 += GroupMax::kBatch) {
    if (threadIdx.x == 0) sh.n_groups = 0;
    __syncthreads();
    groups.each(g0, [&](int i, float top) {
      if (distance(wt.m, top) <= hi) sh.group[atomicAdd(&sh.n_groups, 1u)] = (uint16_t)i;
    });
    __syncthreads();
    // each listed group holds a token at least
    const uint32_t listed = sh.n_groups;
    if (listed > max_groups || have + listed > kCap) return kCap + 1;
    const int items = (int)listed * kVec;
    int next_v[kItems];
    u32x4_t next[kItems];
    auto fetch = [&](int b0) {
#pragma unroll
      for (int l = 0; l < kItems; ++l) {
        const int i = b0 + (int)threadIdx.x + l * kRowThreads;
        next_v[l] = row.nvec;
        if (i < items) {
          const int g = g0 + sh.group[i / kVec];
          next_v[l] = g / kThreads * (kThreads * kVec) + (i % kVec) * kThreads + g % kThreads;
        }
        next[l] = u32x4_t{0, 0, 0, 0};
        if (row.full(next_v[l])) next[l] = row.raw(next_v[l]);
      }
    };
    fetch(0);
    for (int b0 = 0; b0 < items; b0 += kItems * kRowThreads) {
      float z[kItems][R::VE];
      int v[kItems];
#pragma unroll
      for (int l = 0; l < kItems; ++l) {
        v[l] = next_v[l];
        row.take(v[l], next[l], z[l]);
      }
      fetch(b0 + kItems * kRowThreads);  // waits behind this round's work
      // places for all of the wavefront's hits at once
      uint32_t in = 0;
#pragma unroll
      for (int l = 0; l < kItems; ++l)
#pragma unroll
        for (int q = 0; q < R::VE; ++q) {
          const float x = z[l][q];
          in |= (x != kNegInf && distance(wt.m, x) <= hi ? 1u : 0u) << (l * R::VE + q);
        }
      const uint32_t c = __builtin_popcount(in);
      const uint32_t run = (uint32_t)wave_scan(c);
      uint32_t at = 0;
      if ((threadIdx.x & 63) == 63) at = atomicAdd(&sh.n, run);
      at = (uint32_t)__builtin_amdgcn_readlane((int)at, 63) + run - c;
#pragma unroll
      for (int l = 0; l < kItems; ++l) {
        const uint32_t e = (uint32_t)row.first(v[l]);
#pragma unroll
        for (int q = 0; q < R::VE; ++q) {
          if ((in >> (l * R::VE + q)) & 1u) {
            if (at < kCap) sh.list[at] = Entry{__float_as_uint(z[l][q]), e + q, 0};
            ++at;
          }
        }
      }
    }
    __syncthreads();
    have = sh.n;  // not added to before the next batch's second barrier
    if (have > kCap) return have;
  }
  // the weights last, when every thread has its share of them
  for (uint32_t i = threadIdx.x; i < have; i += kRowThreads)
    sh.list[i] = entry_of<DT>(wt, __uint_as_float(sh.list[i].key), sh.list[i].idx);
  __syncthreads();
  return have;
}

struct Drawn {
  int64_t token;
  u64 total;  // weight of all kept tokens
  // the threshold: kept are the keys above tau, and of key tau the tokens up
  // to index last
  uint32_t tau, last;
};

// Draws from the list of candidates, which holds every token the filters can
// keep; `mass` is the weight that top-p refers to without top-k.  With
// `threshold` the list holds one bin of the histogram, `above` is the weight (for
// top-k the number) before it, and only the threshold is taken, of one of the two.
template <int DT>
__device__ __forceinline__ Drawn draw_list(const Ask& a, const Weights& wt, int64_t V, uint32_t n,
                                           u64 mass, bool threshold, u64 above, PickShared& sh) {
  const uint32_t t = threadIdx.x;
  Drawn d;
  d.token = 0;
  d.total = 0;
  d.tau = 0;
  d.last = 0xffffffffu;
  if (n <= kRank && !threshold) {
    // one candidate per lane of the first wavefront: its rank and the weight ranked
    // before it
    const bool mine = t < n;
    const Entry e = mine ? sh.list[t] : Entry{0, 0, 0};
    const u64 q = e.q & ~kKeptBit;
    const uint32_t n_wave = t < 64 ? n : 0;
    // four entries at a time, the last ones filled up with none
    if (t < 4) sh.list[n + t] = Entry{0, 0xffffffffu, 0};
    __syncthreads();
    uint32_t rank = 0;
    u64 before = 0;
    for (uint32_t j = 0; j < n_wave; j += 4) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const Entry o = sh.list[j + i];
        const bool better = o.key > e.key || (o.key == e.key && o.idx < e.idx);
        rank += better;
        before += better ? o.q & ~kKeptBit : 0;
      }
    }
    bool keep = mine && (!a.has_k || rank < (uint32_t)a.k);
    if (a.has_p) {
      if (a.has_k) mass = block_sum(keep ? q : 0, sh);
      keep = keep && (rank == 0 || (double)before < a.p * (double)mass);
    }
    keep = keep && (e.q & kKeptBit);
    d.total = block_sum(keep ? q : 0, sh);  // a barrier: the list has been read
    if (mine) sh.list[t].q = keep ? q : 0;
    if (t == 0) sh.out[0] = 0;
    __syncthreads();
    u64 upto = 0;
    for (uint32_t j = 0; j < n_wave; j += 4) {
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        const Entry o = sh.list[j + i];
        upto += o.idx <= e.idx ? o.q : 0;
      }
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
  // keys count from the least one: fewer bits to select by, and the first nine
  // tell the candidates apart (equal digits queue at one LDS address)
  uint32_t key0 = 0xffffffffu, key1 = 0;
  for (uint32_t i = t; i < n; i += kRowThreads) {
    key0 = min(key0, sh.list[i].key);
    key1 = max(key1, sh.list[i].key);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    key0 = min(key0, (uint32_t)__shfl_xor((int)key0, off, 64));
    key1 = max(key1, (uint32_t)__shfl_xor((int)key1, off, 64));
  }
  __syncthreads();
  if ((t & 63) == 0) sh.wave[t >> 6] = ((u64)key1 << 32) | key0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowWaves; ++i) {
    key0 = min(key0, (uint32_t)sh.wave[i]);
    key1 = max(key1, (uint32_t)(sh.wave[i] >> 32));
  }
  const int key_bits = key1 > key0 ? 32 - __builtin_clz(key1 - key0) : 1;
  const int idx_bits = 64 - __builtin_clzll((u64)V);
  u64 ties = ~(u64)0;  // none: no threshold
  uint32_t tau = 0, last = 0xffffffffu;
  for (int stage = 0; stage < (threshold ? 3 : 4); ++stage) {
    double goal = 0.0;
    if (stage == 0) {  // top-k
      if (!a.has_k) continue;
      if ((u64)a.k - above >= n) {
        if (threshold) tau = key0;  // all of the bin, nothing behind it
        continue;
      }
      goal = (double)((u64)a.k - above);
    } else if (stage == 1) {  // top-p
      if (!a.has_p) continue;
      if (a.has_k) {
        u64 v = 0;
        for (uint32_t i = t; i < n; i += kRowThreads)
          if (ties == ~(u64)0 || sh.list[i].key > tau) v += sh.list[i].q & ~kKeptBit;
        mass = block_sum(v, sh);
        if (ties != ~(u64)0) mass += ties * wt.all(key_value<DT>(tau));
      }
      goal = a.p * (double)mass - (double)above;
    } else if (stage == 2) {  // the last tie kept, where not all are
      if (ties == ~(u64)0) continue;
      u64 c = 0;
      for (uint32_t i = t; i < n; i += kRowThreads) c += sh.list[i].key == tau;
      c = block_sum(c, sh);
      if (ties >= c) continue;
      if (c <= kRank) {
        // few: their indexes side by side, and the rank of each by counting
        uint32_t* idx = reinterpret_cast<uint32_t*>(sh.hist);
        if (t == 0) sh.n = 0;
        __syncthreads();
        for (uint32_t i = t; i < n; i += kRowThreads)
          if (sh.list[i].key == tau) idx[atomicAdd(&sh.n, 1u)] = sh.list[i].idx;
        __syncthreads();
        if (t < c) {
          const uint32_t mine = idx[t];
          uint32_t before = 0;
          for (uint32_t i = 0; i < c; ++i) before += idx[i] < mine;
          if (before == ties - 1) sh.out[0] = mine;
        }
        __syncthreads();
        last = (uint32_t)sh.out[0];
        continue;
      }
      goal = (double)ties;
    } else {  // the token
      u64 v = 0;
      for (uint32_t i = t; i < n; i += kRowThreads) {
        const Entry e = sh.list[i];
        if ((e.q & kKeptBit) && (e.key > tau || (e.key == tau && e.idx <= last)))
          v += e.q & ~kKeptBit;
      }
      d.total = block_sum(v, sh);
      goal = (double)a.u * (double)d.total;
    }
    Sel s = radix_select(stage < 2 ? key_bits : idx_bits, goal, stage == 3, sh, [&](auto f) {
      for (uint32_t i = t; i < n; i += kRowThreads) {
        const Entry e = sh.list[i];
        const bool in = stage == 0   ? true
                        : stage == 1 ? e.key >= tau
                        : stage == 2 ? e.key == tau
                                     : (e.q & kKeptBit) &&
                                           (e.key > tau || (e.key == tau && e.idx <= last));
        const u64 w = stage == 1 || stage == 3 ? e.q & ~kKeptBit : (u64)1;
        if (in) f(stage < 2 ? e.key - key0 : (uint32_t)(V - 1 - e.idx), w);
      }
    });
    if (stage < 2) s.key += key0;
    if (stage == 0) {
      tau = s.key;
      ties = (u64)a.k - above - s.above;
    } else if (stage == 1) {
      u64 c = 0;
      for (uint32_t i = t; i < n; i += kRowThreads) c += sh.list[i].key == s.key;
      c = block_sum(c, sh);
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
  d.last = last;
  return d;
}

// The first token of a segment at which the running sum of amount(index, z),
// from `before` on, exceeds the goal: 64 consecutive vectors are a chunk; the
// chunk of the crossing is found from their sums, the vector and the token in
// it by one wavefront.
template <int DT, class Amount>
__device__ __forceinline__ int64_t pick_in_segment(const Row<DT>& row, int seg, u64 before,
                                                   double goal, Scratch& sh, Amount amount) {
  typedef Row<DT> R;
  typedef Group<DT, kRowThreads> G;
  constexpr int kVec = G::kVec;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int c0 = seg * (kSeg / R::VE);
  __syncthreads();  // the scratch may still be read
  {
    float z[kVec][R::VE];
    G group;
    group.load(row, c0 + t);
    group.get(row, c0 + t, z);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const int64_t e = row.first(c0 + t + j * kRowThreads);
      u64 s = 0;
#pragma unroll
      for (int q = 0; q < R::VE; ++q) s += amount(e + q, z[j][q]);
      s = wave_sum(s);
      if (lane == 0) sh.hist[j * kRowWaves + wave] = s;
    }
  }
  __syncthreads();
  const u64 mine = lane < kVec * kRowWaves ? sh.hist[lane] : 0;
  const u64 run = wave_scan(mine);
  const uint64_t hit = __ballot(mine != 0 && (double)(before + run) > goal);
  const int chunk = hit ? __builtin_ctzll(hit) : 0;
  before += lane64(run - mine, chunk);
  if (t == 0) sh.out[0] = 0;
  if (wave == 0) {
    const int v = c0 + chunk * 64 + lane;
    u64 w[R::VE], s = 0;
#pragma unroll
    for (int q = 0; q < R::VE; ++q) w[q] = 0;
    if (v < row.nvec) {
      float z[R::VE];
      row.load(v, z);
#pragma unroll
      for (int q = 0; q < R::VE; ++q) {
        w[q] = amount(row.first(v) + q, z[q]);
        s += w[q];
      }
    }
    const u64 upto = before + wave_scan(s);
    const uint64_t h = __ballot(s != 0 && (double)upto > goal);
    if (h && lane == __builtin_ctzll(h)) {
      u64 c = upto - s;
      int64_t token = -1;
#pragma unroll
      for (int q = 0; q < R::VE; ++q) {
        c += w[q];
        if (token < 0 && w[q] != 0 && (double)c > goal) token = row.first(v) + q;
      }
      sh.out[0] = (u64)token;
    }
  }
  __syncthreads();
  return (int64_t)sh.out[0];
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

// Draws row r, or leaves it to sample_rest_kernel.
template <int DT>
__device__ __forceinline__ void pick_row(const SampleParams& p, const Row<DT>& row, const Ask& a,
                                         int64_t r, PickShared& sh) {
  typedef Row<DT> R;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  GroupMax groups;
  groups.init(p.group_max + r * p.segs * kThreads, p.segs);
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
  const Weights wt = weights_of(p, a, m);
  if (a.greedy || a.plain()) {
    // the segment that holds the token: the first with the maximum, or the one
    // in which the running sum crosses; every wavefront finds it
    u64 total = 0, before = 0;
    double goal = 0.0;
    if (!a.greedy) {
      if (a.small(p.V)) {
        for (int i = t; i < row.nvec; i += kRowThreads) {
          float z[R::VE];
          row.load(i, z);
#pragma unroll
          for (int j = 0; j < R::VE; ++j) total += wt.all(z[j]);
        }
        total = block_sum(total, sh);
      } else {
        for (int i = lane; i < p.segs; i += 64) total += get_shared(&p.seg_sum[r * p.segs + i]);
        total = wave_sum(total);
      }
      goal = (double)a.u * (double)total;
    }
    int seg = 0;
    // a small row is one segment
    for (int i = 0; i < p.segs && !a.small(p.V); i += 64) {
      u64 v = 0;
      if (i + lane < p.segs)
        v = a.greedy ? (u64)(seg_max[i + lane] == m)
                     : get_shared(&p.seg_sum[r * p.segs + i + lane]);
      const u64 run = wave_scan(v);
      const uint64_t hit = __ballot(v != 0 && (double)(before + run) > goal);
      if (hit) {
        const int who = __builtin_ctzll(hit);
        seg = i + who;
        before += lane64(run - v, who);
        break;
      }
      before += lane64(run, 63);
    }
    const int64_t token = pick_in_segment<DT>(row, seg, before, goal, sh, [&](int64_t, float z) {
      const u64 q = wt.all(z);
      return a.greedy ? (u64)(z == m) : q;
    });
    if (t == 0) write_out<DT>(p, r, row, a, m, token, total);
    return;
  }
  // candidates: distances up to hi
  float hi = __builtin_huge_valf();
  u64 mass = 0;
  SampleState st{kRow, 0.0f, 0.0f, 0, 0, 0};
  if (a.has_k || a.has_p) {
    // the bin of the distance where the count or the mass is reached, 4 bins a
    // thread: of the row's histogram (made here for a small row), or of the group
    // maxima (k groups with maxima of at least the k-th largest hold k tokens as large)
    constexpr int kPer = kBins / kRowThreads;
    u64* bins = reinterpret_cast<u64*>(sh.list);  // the list comes later
    if (a.hist(p.V)) {
      for (int i = t; i < kBins; i += kRowThreads) bins[i] = get_shared(&p.hist[r * kBins + i]);
    } else {
      for (int i = t; i < kBins; i += kRowThreads) bins[i] = 0;
      __syncthreads();
      if (!a.has_k || !a.group_bound(p.V)) {
        for (int i = t; i < row.nvec; i += kRowThreads) {
          float z[R::VE];
          row.load(i, z);
#pragma unroll
          for (int j = 0; j < R::VE; ++j) {
            const u64 q = a.has_k ? (u64)(z[j] != kNegInf) : wt.all(z[j]);
            mass += q;
            if (q != 0) atomicAdd(&bins[bin_of(m, z[j])], q);
          }
        }
        mass = block_sum(mass, sh);
      } else {
        for (int g0 = 0; g0 < groups.n; g0 += GroupMax::kBatch)
          groups.each(g0, [&](int, float g) { atomicAdd(&bins[bin_of(m, g)], (u64)1); });
      }
    }
    if (!a.has_k && !a.small(p.V)) {
      for (int i = lane; i < p.segs; i += 64) mass += get_shared(&p.seg_sum[r * p.segs + i]);
      mass = wave_sum(mass);
    }
    const double goal = a.has_k ? (double)a.k : a.p * (double)mass;
    if (t == 0) {
      sh.out[0] = kBins - 1;  // never reached: all bins
      sh.out[1] = 0;
    }
    __syncthreads();
    u64 v = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) v += bins[t * kPer + j];
    const u64 run = wave_scan(v);
    if (lane == 63) sh.wave[wave] = run;
    __syncthreads();
    u64 before = run - v;
    for (int i = 0; i < wave; ++i) before += sh.wave[i];
    if (!reached(before, goal, false) && reached(before + v, goal, false)) {
      for (int j = 0; j < kPer; ++j) {
        const u64 w = bins[t * kPer + j];
        if (reached(before + w, goal, false)) {
          sh.out[0] = t * kPer + j;
          sh.out[1] = before;
          break;
        }
        before += w;
      }
    }
    __syncthreads();
    const uint32_t bin = (uint32_t)sh.out[0];
    // the distances of bin b lie between bits (base + b) << 16 and the next
    if (bin < kBins - 1) hi = __uint_as_float(((kBinBase + bin + 1) << 16) - 1);
    // the threshold lies in this bin, unless top-p follows a top-k
    if (!a.has_k || (!a.has_p && a.hist(p.V))) {
      st.what = kThreshold;
      st.lo = bin > 0 ? __uint_as_float((kBinBase + bin) << 16) : 0.0f;
      st.hi = hi;
      st.above = sh.out[1];
      st.mass = mass;
    }
  } else {
    // min-p alone: T ln(1 / min_p) and what its rounding, or a weight's (1e-12 covers its error
    // of 4e-14, and the tokens that weigh 1 in FP64 beside the maxima), may leave out
    hi = (float)((double)a.T * (1e-12 - log(a.minp) * (1.0 + 1e-6))) + 1e-30f;
    hi += hi * 1e-6f;
    // nothing but min-p: every token that it can keep lies before the bin, and none in it.
    // A bound beyond FP32 bounds nothing, nor do the distances that overflow with it: NaN,
    // before which every token lies
    st.what = kThreshold;
    st.lo = hi < __builtin_huge_valf() ? hi : __builtin_nanf("");
    st.hi = -1.0f;
  }
  // rows that other kernels can finish over all segments gather little here, those
  // that cannot fit nothing
  const uint32_t most = a.has_k ? (a.k > kCap ? 0 : kCap) : st.what == kThreshold ? 512 : kCap;
  const uint32_t n = gather_groups<DT>(row, groups, wt, hi, a.small(p.V) ? kCap : most, sh);
  if (n > kCap) {
    // (a call without state has rows of at most kCap tokens, which always fit)
    if (t == 0 && p.state) p.state[r] = st;
    return;
  }
  const Drawn d = draw_list<DT>(a, wt, p.V, n, mass, false, 0, sh);
  if (t == 0) write_out<DT>(p, r, row, a, m, d.token, d.total);
}

// A row per workgroup, or JOINED with sample_mass_kernel a segment per workgroup, the
// last of a row's drawing.
template <int DT, bool JOINED>
__global__ __launch_bounds__(kRowThreads, 4) void sample_pick_kernel(SampleParams p) {
  __shared__ PickShared sh;
  int64_t r = blockIdx.x;
  int seg = 0;
  if (JOINED && !row_and_segment(p, &r, &seg)) return;
  const Ask a = ask_of(p, r);
  const Row<DT> row = row_of<DT>(p, r);
  if (JOINED) {
    if (needs_mass(a, p.V)) {
      mass_of_segment<DT, kRowThreads>(p, row, a, r, seg, reinterpret_cast<u64*>(sh.list),
                                       sh.wave);
      if (!last_of_row(p.done + 2 * r, p.segs, sh)) return;
    } else if (seg != 0) {
      return;
    }
  }
  pick_row<DT>(p, row, a, r, sh);
}

// Rows whose candidates do not fit in LDS, one segment each: the kept weight of
// the tokens before the histogram's bin, and the bin's tokens appended to the
// row's list (over its histogram, which has been read).
template <int NT>
struct KeepShared {
  float low[NT / 64][64 * (kSeg / NT)];  // a wavefront's tokens before the bin, side by side
  u64 part[NT / 64];
  uint32_t cnt[NT / 64], base;
};

template <int DT, int NT>
__device__ __forceinline__ void keep_segment(const SampleParams& p, const Row<DT>& row,
                                             const Ask& a, int64_t r, int seg, KeepShared<NT>& sh) {
  typedef Row<DT> R;
  typedef Group<DT, NT> G;
  constexpr int kVec = G::kVec, kTokens = kVec * R::VE;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int v0 = seg * (kSeg / R::VE) + t;
  G group;
  group.load(row, v0);
  const Weights wt = weights_of(p, a, row_max(p.seg_max + r * p.segs, p.segs));
  const float lo = p.state[r].lo, hi = p.state[r].hi;
  float z[kVec][R::VE];
  group.get(row, v0, z);
  // bit j: token j is in the bin, or before it
  uint32_t in = 0, low = 0;
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    const float v = z[j / R::VE][j % R::VE], d = distance(wt.m, v);
    in |= (v != kNegInf && d >= lo && d <= hi ? 1u : 0u) << j;
    low |= (!(d >= lo) ? 1u : 0u) << j;
    if (j % 8 == 7) __builtin_amdgcn_sched_barrier(0);
  }
  // The weights are what takes time: first the tokens before the bin move together, so that
  // every lane forms one (256 rows of top-p 0.9: a weight for every token 48 us, for these
  // 31; four at a time instead of two spilled and took 38).
  float* mine = sh.low[wave];
  const uint32_t n_low = __builtin_popcount(low), run_low = (uint32_t)wave_scan(n_low);
  const int all_low = __builtin_amdgcn_readlane((int)run_low, 63);
  uint32_t to = run_low - n_low;
#pragma unroll
  for (int j = 0; j < kTokens; ++j) {
    if ((low >> j) & 1u) mine[to++] = z[j / R::VE][j % R::VE];
    if (j % 8 == 7) __builtin_amdgcn_sched_barrier(0);
  }
  __syncthreads();
  u64 s = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < all_low; i0 += 2 * 64) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = i0 + 64 * j + lane;
      const u64 q = wt.kept(mine[min(i, all_low - 1)]);
      s += i < all_low ? q : 0;
    }
  }
  s = wave_sum(s);
  const uint32_t c = __builtin_popcount(in);
  const uint32_t run = (uint32_t)wave_scan(c);
  if (lane == 63) sh.cnt[wave] = run;
  if (lane == 0) sh.part[wave] = s;
  __syncthreads();
  uint32_t n = 0, at = run - c;
#pragma unroll
  for (int i = 0; i < NT / 64; ++i) {
    at += i < wave ? sh.cnt[i] : 0;
    n += sh.cnt[i];
  }
  if (t == 0) {
    s = 0;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) s += sh.part[i];
    put_shared(&p.seg_sum[r * p.segs + seg], s);
    sh.base = n ? atomicAdd(&p.state[r].n, n) : 0;
  }
  __syncthreads();
  at += sh.base;
  uint32_t* list = reinterpret_cast<uint32_t*>(p.hist + r * kBins);
  for (; in; in &= in - 1, ++at) {
    const int j = __builtin_ctz(in);
    if (at < kCap)
      put_shared(&list[at], (uint32_t)(row.first(v0 + (j / R::VE) * NT) + j % R::VE));
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads, 4) void sample_kept_kernel(SampleParams p) {
  __shared__ KeepShared<kThreads> sh;
  int64_t r;
  int seg;
  if (!row_and_segment(p, &r, &seg)) return;
  if (p.state[r].what != kThreshold) return;
  keep_segment<DT, kThreads>(p, row_of<DT>(p, r), ask_of(p, r), r, seg, sh);
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
      for (uint32_t i = threadIdx.x; i < n_list; i += kRowThreads)
        f(__uint_as_float(sh.key[i]), (int64_t)sh.idx[i]);
    } else {
      row.each(0, row.nvec, threadIdx.x, kRowThreads, [&](int64_t e, const float* z) {
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
        row.each(0, row.nvec, threadIdx.x, kRowThreads, [&](int64_t, const float* z) {
#pragma unroll
          for (int j = 0; j < R::VE; ++j)
            if (R::key(z[j]) > tau) v += wt.all(z[j]);
        });
        mass_k = block_sum(v, sh) + ties * wt.all(key_value<DT>(tau));
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
    n = block_sum(n, sh);
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

// A row per workgroup, or JOINED with sample_kept_kernel a segment per workgroup.
template <int DT, bool JOINED>
__global__ __launch_bounds__(kRowThreads, 4) void sample_rest_kernel(SampleParams p) {
  __shared__ union {
    PickShared pick;
    Shared row;
    KeepShared<kRowThreads> keep;
  } both;
  typedef Row<DT> R;
  int64_t r = blockIdx.x;
  int seg = 0;
  if (JOINED && !row_and_segment(p, &r, &seg)) return;
  const uint32_t what = p.state[r].what;
  if (what == kDone || (what == kRow && seg != 0)) return;
  const Ask a = ask_of(p, r);
  const R row = row_of<DT>(p, r);
  if (JOINED && what == kThreshold) {
    keep_segment<DT, kRowThreads>(p, row, a, r, seg, both.keep);
    if (!last_of_row(p.done + 2 * r + 1, p.segs, both.pick)) return;
  }
  const float m = row_max(p.seg_max + r * p.segs, p.segs);
  const Weights wt = weights_of(p, a, m);
  SampleState st = p.state[r];
  st.n = get_shared(&p.state[r].n);
  Drawn d;
  if (st.what == kRow || st.n > kCap || p.segs > kKeepSegs) {
    d = draw_row<DT>(row, a, wt, both.row);
  } else {
    PickShared& sh = both.pick;
    const int t = threadIdx.x, lane = t & 63;
    const u64* sum = (const u64*)p.seg_sum + r * p.segs;
    const uint32_t* list = reinterpret_cast<const uint32_t*>(p.hist + r * kBins);
    for (uint32_t i = t; i < st.n; i += kRowThreads) {
      const uint32_t idx = get_shared(&list[i]);
      float z;
      if constexpr (DT == 0)
        z = reinterpret_cast<const float*>(row.base)[idx] + 0.0f;
      else
        z = from_bf16(reinterpret_cast<const uint16_t*>(row.base)[idx]) + 0.0f;
      sh.list[i] = entry_of<DT>(wt, z, idx);
    }
    __syncthreads();
    d.tau = 0;
    d.last = 0xffffffffu;
    if (st.n > 0) d = draw_list<DT>(a, wt, p.V, st.n, st.mass, true, st.above, sh);
    // what a segment keeps: its sum before the bin and its share of the list
    __syncthreads();
    u64* keep = sh.keep;
    for (int i = t; i < p.segs; i += kRowThreads) keep[i] = get_shared(&sum[i]);
    __syncthreads();
    for (uint32_t i = t; i < st.n; i += kRowThreads) {
      const Entry e = sh.list[i];
      if ((e.q & kKeptBit) && (e.key > d.tau || (e.key == d.tau && e.idx <= d.last)))
        atomicAdd(&keep[(e.idx + (uint32_t)row.off) / kSeg], e.q & ~kKeptBit);
    }
    __syncthreads();
    u64 total = 0;
    for (int i = lane; i < p.segs; i += 64) total += keep[i];
    total = wave_sum(total);
    const double goal = (double)a.u * (double)total;
    u64 before = 0;
    seg = 0;
    for (int i = 0; i < p.segs; i += 64) {
      const u64 v = i + lane < p.segs ? keep[i + lane] : 0;
      const u64 run = wave_scan(v);
      const uint64_t hit = __ballot(v != 0 && (double)(before + run) > goal);
      if (hit) {
        const int who = __builtin_ctzll(hit);
        seg = i + who;
        before += lane64(run - v, who);
        break;
      }
      before += lane64(run, 63);
    }
    d.total = total;
    d.token = pick_in_segment<DT>(row, seg, before, goal, sh, [&](int64_t i, float z) -> u64 {
      const uint32_t k = R::key(z);
      const u64 q = wt.kept(z);
      return distance(m, z) < st.lo || k > d.tau || (k == d.tau && i <= (int64_t)d.last) ? q : 0;
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

bool sample_size_ok(int64_t N, int64_t V) {
  return N < ((int64_t)1 << 22) && V <= ((int64_t)1 << 28) &&
         N * segments(V) < ((int64_t)1 << 31);
}

// Rows of at most kCap tokens are served by sample_max_kernel and sample_pick_kernel alone:
// they need no sums, histogram, state or counters.
size_t sample_workspace_bytes(int64_t N, int64_t V) {
  const size_t rows = (size_t)N, s = rows * (size_t)segments(V);
  const size_t maxima = 256 + up256(s * kThreads * 4) + up256(s * 4);
  if (V <= kCap) return maxima;
  return maxima + up256(s * 8) + up256(rows * kBins * 8) + up256(rows * sizeof(SampleState)) +
         up256(rows * 8);
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
  p.group_max = reinterpret_cast<float*>(take(s * kThreads * 4));
  p.seg_max = reinterpret_cast<float*>(take(s * 4));
  const bool mass = p.V > kCap;
  if (mass) {
    p.seg_sum = reinterpret_cast<unsigned long long*>(take(s * 8));
    p.hist = reinterpret_cast<unsigned long long*>(take(rows * kBins * 8));
    p.state = reinterpret_cast<SampleState*>(take(rows * sizeof(SampleState)));
    p.done = reinterpret_cast<uint32_t*>(take(rows * 8));
  }
  p.rows = (uint32_t)N;
  const dim3 seg_grid = grid2(N * p.segs);
  // without filters no row has candidates
  const bool rest = mass && (p.top_k || p.top_p || p.min_p);
  const bool joined = mass && N * p.segs <= kJoined;
  p.has = (p.temperature ? SampleParams::kT : 0) | (p.top_k ? SampleParams::kK : 0) |
          (p.top_p ? SampleParams::kP : 0) | (p.min_p ? SampleParams::kM : 0);
  if (!p.temperature) p.temperature = p.u;
  if (!p.top_k) p.top_k = reinterpret_cast<const int32_t*>(p.u);
  if (!p.top_p) p.top_p = p.u;
  if (!p.min_p) p.min_p = p.u;
  p.inv_v = 1.0 / (double)p.V;
  if (!rest) p.state = nullptr;
  auto run = [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    hipLaunchKernelGGL((sample_max_kernel<DT>), seg_grid, dim3(kThreads), 0, stream, p);
    if (joined) {
      hipLaunchKernelGGL((sample_pick_kernel<DT, true>), seg_grid, dim3(kRowThreads), 0, stream,
                         p);
      if (rest)
        hipLaunchKernelGGL((sample_rest_kernel<DT, true>), seg_grid, dim3(kRowThreads), 0,
                           stream, p);
      return;
    }
    if (mass)
      hipLaunchKernelGGL((sample_mass_kernel<DT>), seg_grid, dim3(kThreads), 0, stream, p);
    hipLaunchKernelGGL((sample_pick_kernel<DT, false>), dim3((unsigned)N), dim3(kRowThreads), 0,
                       stream, p);
    if (rest) {
      hipLaunchKernelGGL((sample_kept_kernel<DT>), seg_grid, dim3(kThreads), 0, stream, p);
      hipLaunchKernelGGL((sample_rest_kernel<DT, false>), dim3((unsigned)N), dim3(kRowThreads),
                         0, stream, p);
    }
  };
  if (dtype == 0)
    run(std::integral_constant<int, 0>{});
  else
    run(std::integral_constant<int, 1>{});
  return hipGetLastError();
}

}  // namespace vce
