// The matrix-core building block of the linear forms: C[i][j] = sum_k P(i, k) Q(j, k) over
// BF16 operands in 256 x 256 output tiles, each tile finished by an epilogue of the
// including file's choice.  Design and measurements: lce_kernels.hip.
#pragma once

#include <type_traits>

#include "vce_device.h"
#include "vce_internal.h"

namespace vce {

namespace {

constexpr int BM = 256;   // output rows per tile (P side)
constexpr int BN = 256;   // output cols per tile (Q side)
constexpr int BK = 64;    // K slice per stage
constexpr int NT = 256;   // threads per workgroup: 4 wavefronts, one per SIMD
constexpr int WM = 128;   // output rows per wavefront
constexpr int WN = 128;   // output cols per wavefront
constexpr int NA = WM / 32;                        // 32-row blocks per wavefront (4)
constexpr int NB = WN / 32;                        // 32-column blocks per wavefront (4)
constexpr int NWC = BN / WN;                       // wavefronts across the columns (2)
constexpr int UNITS = BM * BK * 2 / 1024;          // 1 KB units per operand per slice (32)
constexpr int UPW = UNITS / (NT / 64);             // units per wave per operand (8)
constexpr int GROUP_I = 8;                         // row tiles per band of the tile order
constexpr uint32_t kOob = 0x80000000u;             // buffer offset that reads as 0
constexpr int kSmemElems = 2 * (BM + BN) * BK;  // two stages of both operands (128 KB)

static_assert(BM == BN, "one loader shape serves both operands");
static_assert(NA == 4 && NB == 4 && UPW == 8, "the schedule below assumes these");

#define LDS_AS __attribute__((address_space(3)))

// An operand of C[i][j] = sum_k P(i, k) Q(j, k), BF16:
//   K-contiguous   (DIM = false): element (d, k) at base[d * ld + k]
//   dim-contiguous (DIM = true):  element (d, k) at base[k * ld + d]
// Reads with d >= dim_limit or k >= k_limit return 0.  Along the contiguous
// axis the test is per 8-element chunk (its first element), so a buffer must
// hold zeros from its limit on that axis up to the next multiple of 8.
struct Operand {
  const uint16_t* base;
  int64_t ld;
  int64_t dim_limit;
  int64_t k_limit;
};

// LDS stage of one operand (256 x 64 elements, 32 KB, 32 units of 1 KB):
//  * K-contiguous: 256 rows (d) of 64 k (128 B, eight 16-byte chunks);
//    logical chunk c of row d sits at c ^ swz(d).
//  * dim-contiguous: two halves (d < 128, d >= 128) of 64 rows (k) of 128 d
//    (256 B, sixteen chunks); logical chunk c of row k sits at c ^ 4 (k & 3).
// Both make the fragment reads below bank-conflict free (measured: a
// transposed read serves 32 lanes, 4 rows x 64 B, per 256-byte bank cycle,
// so the four rows must fall in different 64-byte quarters).
__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

// Moves one operand's 256 x 64 slices in 1 KB units, 8 per wave: unit q =
// 8 w + i of wave w, lane l, 16 bytes each.  All that varies with i is a
// scalar offset of the global read and an immediate (or one XOR) of the LDS
// write, so a loader holds two VGPRs:
//  * K-contiguous: rows 8 q .. 8 q + 7, lane l reads logical chunk l % 8 of
//    row 8 q + l / 8 and writes it at physical chunk (l % 8) ^ swz(row) =
//    (l % 8) ^ (l / 8) ^ i.  Rows past dim_limit are cut off by the buffer
//    size; with MASK, chunks at or past k_limit by an out-of-range offset.
//  * dim-contiguous: half q / 16 (= w / 2), k rows 4 (q % 16) + l / 16, lane
//    chunk l % 16 read from logical chunk (l % 16) ^ 4 (l / 16 % 4) of that
//    row and written at 16 l of the unit.  Columns past dim_limit get an
//    out-of-range offset; k rows past k_limit are cut off by the buffer size.
// at(k0) gives the slice's buffer (scalar, once per slice); get() loads a
// unit into registers, put() writes registers to the stage; direct() loads a
// unit of the first slice straight into LDS (the prologue).
struct SliceRef {
  __amdgpu_buffer_rsrc_t rs;
  int nv;  // K-contiguous with MASK: chunks (of 8 k) of the slice below k_limit, 0..8
};

template <bool DIM>
struct SliceLoader {
  const uint16_t* tbase;  // operand at the tile's first element, k = 0
  int64_t ld;
  int64_t k_limit;
  int64_t rows_bytes;  // K-contiguous: bytes of the tile's rows below dim_limit
  uint32_t voff;       // this lane's byte offset in unit 0, or kOob
  uint32_t ustep;      // bytes between the sources of consecutive units
  int lds;             // element offset of this lane's 16 bytes of unit 0 in a stage
  int kch;             // K-contiguous: the logical chunk this lane reads (l % 8)
  __device__ __forceinline__ void init(const Operand& op, int64_t d0, int wave, int lane) {
    k_limit = op.k_limit;
    ld = op.ld;
    if (!DIM) {
      tbase = op.base + d0 * op.ld;
      const int64_t rl = op.dim_limit - d0;
      rows_bytes = rl <= 0 ? 0 : rl * op.ld * 2;
      const int row = 8 * UPW * wave + (lane >> 3);
      voff = (uint32_t)(row * op.ld * 2 + (lane & 7) * 16);
      ustep = (uint32_t)__builtin_amdgcn_readfirstlane((int)(8 * op.ld * 2));
      kch = lane & 7;
      const int c0 = ((lane & 7) ^ (lane >> 3)) & 7;  // physical chunk in unit 0
      lds = row * BK + c0 * 8;                        // unit i: (lds ^ 8 i) + 512 i
    } else {
      tbase = op.base + d0;
      rows_bytes = 0;
      const int krow = 32 * (wave & 1) + (lane >> 4);
      const int c = (lane & 15) ^ (4 * ((lane >> 4) & 3));
      const int d = 128 * (wave >> 1) + 8 * c;
      voff = (d0 + d < op.dim_limit) ? (uint32_t)(krow * op.ld * 2 + d * 2) : kOob;
      ustep = (uint32_t)__builtin_amdgcn_readfirstlane((int)(4 * op.ld * 2));
      kch = 0;
      lds = 512 * UPW * wave + 8 * lane;  // unit i: + 512 i
    }
  }
  // the slice starting at k0 (a multiple of BK, possibly past K).  MASK:
  // reads at or past k_limit give 0.  Without it K is a multiple of 2 BK and
  // the caller clamps slices past the end (prefetched, never used) to the
  // last one.
  template <bool MASK>
  __device__ __forceinline__ SliceRef at(int64_t k0) const {
    SliceRef r;
    r.nv = 8;
    const int64_t kb = k0;
    if (!DIM) {
      r.rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint16_t*>(tbase + kb), (short)0,
          rows_bytes > 0x7fffffff ? 0x7fffffff : (int)rows_bytes, 0x00020000);
      if (MASK) {
        const int64_t left = k_limit - k0;
        r.nv = left <= 0 ? 0 : (left >= BK ? 8 : (int)((left + 7) >> 3));
      }
    } else {
      int64_t bytes = 0x7fffffff;
      if (MASK) {
        const int64_t left = k_limit - k0;
        bytes = left <= 0 ? 0 : left * ld * 2;
        if (bytes > 0x7fffffff) bytes = 0x7fffffff;
      }
      r.rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(tbase + kb * ld), (short)0,
                                               (int)bytes, 0x00020000);
    }
    return r;
  }
  template <bool MASK>
  __device__ __forceinline__ u32x4_t get(const SliceRef& r, int i) const {
    // K-contiguous: this lane reads logical chunk l % 8, which lies below
    // k_limit iff (l % 8) < nv
    const uint32_t o = (!MASK || DIM || kch < r.nv) ? voff : kOob;
    return __builtin_bit_cast(
        u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r.rs, o, (int)(i * ustep), 0));
  }
  __device__ __forceinline__ void put(uint16_t LDS_AS* stage, int i, const u32x4_t& v) const {
    const int e = DIM ? lds + 512 * i : (lds ^ (8 * i)) + 512 * i;
    *reinterpret_cast<u32x4_t LDS_AS*>(stage + e) = v;
  }
  // Unit i straight into LDS: lane l fills the 16 bytes at 16 l of the unit,
  // so a K-contiguous lane reads the logical chunk that sits there,
  // (l % 8) ^ (l / 8) ^ i, instead of l % 8.
  template <bool MASK>
  __device__ __forceinline__ void direct(uint16_t LDS_AS* stage, const SliceRef& r, int wave,
                                         int lane, int i) const {
    uint32_t o = voff;
    if (!DIM) {
      const int c = ((lane & 7) ^ (lane >> 3) ^ i) & 7;
      o = voff - (uint32_t)((lane & 7) * 16) + (uint32_t)(c * 16);
      if (MASK && c >= r.nv) o = kOob;
    }
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r.rs, (void LDS_AS*)(stage + 512 * (UPW * wave + i)), 16, o, (int)(i * ustep), 0, 0);
  }
};

typedef short v4i16_t __attribute__((ext_vector_type(4)));

// MFMA operand of the 32 tile rows d0 .. d0 + 31 (d0 a multiple of 32) for
// k-step ks (k = 16 ks .. 16 ks + 15): lane l gets row d0 + l % 32 and the 8 k
// values from 16 ks + 8 (l / 32).
template <bool DIM>
__device__ __forceinline__ bf16x8_t frag(const uint16_t LDS_AS* s, int d0, int ks, int lane) {
  if (!DIM) {
    const int row = d0 + (lane & 31), chunk = 2 * ks + (lane >> 5);
    return __builtin_bit_cast(
        bf16x8_t,
        *reinterpret_cast<const u32x4_t LDS_AS*>(s + row * BK + ((chunk ^ swz(row)) * 8)));
  } else {
    // ds_read_tr16_b64: in each 16-lane group, lane 4 j + q gives the address
    // of 4 elements (q-th quarter) of source row j; lane i receives element i
    // of rows 0..3.  Rows are k here, so lane i gets 4 consecutive k of
    // column d = base + i; two reads give the 8 k values.
    const int g = lane >> 4, j = (lane >> 2) & 3, q = lane & 3;
    const int d = d0 + 16 * (g & 1) + 4 * q;
    const int k = 16 * ks + 8 * (g >> 1) + j;
    const uint16_t LDS_AS* p =
        s + (d >> 7) * 8192 + k * 128 + ((((d & 127) >> 3) ^ (4 * j)) * 8) + (d & 7);
    const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((v4i16_t LDS_AS*)p);
    const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((v4i16_t LDS_AS*)(p + 4 * 128));
    const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
    return __builtin_bit_cast(bf16x8_t, u32x4_t{a[0], a[1], b[0], b[1]});
  }
}

// Hardware workgroup id -> (row tile, col tile).
__device__ __forceinline__ void tile_of(int b, int n_ti, int n_tj, int* ti, int* tj) {
  const int n = n_ti * n_tj;
  const int q = n >> 3, rem = n & 7;
  const int x = b & 7, slot = b >> 3;
  const int t = x * q + (x < rem ? x : rem) + slot;  // contiguous range per XCD
  const int band = t / (GROUP_I * n_tj);
  const int in_band = t - band * GROUP_I * n_tj;
  const int left = n_ti - band * GROUP_I;
  const int gi = left < GROUP_I ? left : GROUP_I;
  *ti = band * GROUP_I + in_band % gi;
  *tj = in_band / gi;
}

// Per-wave state of the main loop.
struct LoopState {
  f32x16_t acc[NA][NB];
  bf16x8_t FA[NA];          // P fragments (refilled for the next k-step as they die)
  bf16x8_t FB[2][NB];       // Q fragments of the current and the next k-step
  u32x4_t R[2][2 * UPW];    // register buffers: units 0..7 of P, 8..15 of Q
};

// Slice k of the main loop (its data in stage k & 1, its first k-step's
// fragments in FA and FB[0]).  During k-steps 0..2 the wave writes slice
// k + 1 from register buffer B1 = (k + 1) & 1 to the other stage and refills
// the buffer with slice k + 3.  The barrier early in k-step 3 (after its
// first two MFMAs, before any read of the other stage) publishes slice k + 1
// (every wave waited for its own writes) and tells that stage k is no longer
// read (every wave's fragments of k-step 3 are in registers), so the next
// round of writes may go there.  MFMAs run a-major: P fragment a dies
// after MFMA 4 a + 3 and is refilled with the next k-step's right then; the
// next Q fragments go to the other buffer after MFMA 1 (MFMA 2 in k-step
// 3, behind the barrier).  Waits: the compiler
// places s_waitcnt vmcnt before each LDS write (its load was issued 32 loads
// earlier) and lgkmcnt before the MFMAs that use fresh fragments.
template <int B1, bool PD, bool QD, bool MASK, bool ZERO = false>
__device__ __forceinline__ void loop_slice(LoopState& S, const SliceLoader<PD>& lp,
                                           const SliceLoader<QD>& lq, uint16_t LDS_AS* sp,
                                           uint16_t LDS_AS* sq, int k, int klast, int wr,
                                           int wc, int lane) {
  constexpr int cur = B1 ^ 1;  // k & 1: the loop runs slices in pairs
  const uint16_t LDS_AS* cp = sp + cur * BM * BK;
  const uint16_t LDS_AS* cq = sq + cur * BN * BK;
  uint16_t LDS_AS* np = sp + (cur ^ 1) * BM * BK;
  uint16_t LDS_AS* nq = sq + (cur ^ 1) * BN * BK;
  const int k3 = MASK || k + 3 < klast ? k + 3 : klast;
  const SliceRef rp = lp.template at<MASK>((int64_t)k3 * BK);
  const SliceRef rq = lq.template at<MASK>((int64_t)k3 * BK);
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) {
    const int f = ks & 1;
#pragma unroll
    for (int a = 0; a < NA; ++a) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int m = a * NB + b;
        // the barrier goes in after two MFMAs of k-step 3 (their operands are
        // in registers), so the MFMA pipe stays busy while the wave waits for
        // its last fragment read and for the other waves
        if (ks == 3 && m == 2) {
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        // ZERO (the tile's first slice): k-step 0 starts from C = 0, an
        // inline constant of the MFMA, so the accumulators need no clearing
        const f32x16_t c = (ZERO && ks == 0) ? f32x16_t{} : S.acc[a][b];
        S.acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(S.FA[a], S.FB[f][b], c, 0, 0, 0);
        // next k-step's Q fragments (at k-step 3: of the next slice, from the
        // stage the barrier has just published)
        if (m == (ks == 3 ? 2 : 1)) {
#pragma unroll
          for (int r = 0; r < NB; ++r)
            S.FB[f ^ 1][r] = ks < 3 ? frag<QD>(cq, wc * WN + 32 * r, ks + 1, lane)
                                    : frag<QD>(nq, wc * WN + 32 * r, 0, lane);
        }
        if (b == NB - 1)
          S.FA[a] = ks < 3 ? frag<PD>(cp, wr * WM + 32 * a, ks + 1, lane)
                           : frag<PD>(np, wr * WM + 32 * a, 0, lane);
        const int pos = ks * 16 + m;
        if (ks < 3 && pos % 3 == 2) {
          const int u = pos / 3;  // 0..15
          if (u < UPW) {
            lp.put(np, u, S.R[B1][u]);
            S.R[B1][u] = lp.template get<MASK>(rp, u);
          } else {
            lq.put(nq, u - UPW, S.R[B1][u]);
            S.R[B1][u] = lq.template get<MASK>(rq, u - UPW);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

// Accumulator register r of block (a, b) of a lane holds
//   row i = i0 + 128 wr + 32 a + 8 (r / 4) + 4 (lane / 32) + r % 4
//   col j = j0 + 128 wc + 32 b + lane % 32
// for wavefront (wr, wc) = (wave / 2, wave % 2).
// One output tile: tile number b of the problem (P, Q, K), then the epilogue.
// MASK: K is not a multiple of 2 BK (or is 0): k is masked on every read.
// Up to three operand pairs whose products one tile sums before its
// epilogue: C[i][j] = sum_s sum_k P_s(i, k) Q_s(j, k), every pair with the
// same K.  One pair is the plain GEMM; three carry the FP32-input form, whose
// operands are each split into two BF16 planes (see split_bf16_kernel).
template <int NSEG>
struct Segs {
  Operand P[NSEG], Q[NSEG];
  // pair s by value (constant indices only, so the kernel arguments are read
  // in place and never copied to scratch)
  __device__ __forceinline__ Operand p(int s) const {
    Operand r = P[0];
#pragma unroll
    for (int t = 1; t < NSEG; ++t)
      if (s == t) r = P[t];
    return r;
  }
  __device__ __forceinline__ Operand q(int s) const {
    Operand r = Q[0];
#pragma unroll
    for (int t = 1; t < NSEG; ++t)
      if (s == t) r = Q[t];
    return r;
  }
};

// One operand pair's sum over K added to the accumulators in S (ZERO: stored
// into them, whatever they held): loaders, prologue and main loop, then a
// drain and a barrier, after which both LDS stages are free again (for the
// next pair or the epilogue).
template <bool PD, bool QD, bool MASK, bool ZERO>
__device__ __forceinline__ void mainloop(LoopState& S, const Operand& P, const Operand& Q,
                                         int64_t K, int64_t i0, int64_t j0, int wave, int lane,
                                         int wr, int wc, uint16_t LDS_AS* sp,
                                         uint16_t LDS_AS* sq) {
  SliceLoader<PD> lp;
  SliceLoader<QD> lq;
  lp.init(P, i0, wave, lane);
  lq.init(Q, j0, wave, lane);
  // Q's stages start 64 KB into LDS, past the 16-bit offset of an LDS
  // instruction; with that base opaque to the compiler, each fragment address
  // of Q is one register for both stages (stage and block go in the offset).
  // Measured on the one-pair tile only (it gave the three-pair tile more
  // spills).
  if (ZERO) asm volatile("" : "+v"(sq));
  // An even number of slices (the loop body runs two); slices at or past K
  // read as zeros and add nothing.
  const int nk = (int)((K + 2 * BK - 1) / (2 * BK)) * 2;
  // last real slice (without MASK, prefetches past it re-read it)
  const int klast = (int)((K + BK - 1) / BK) - 1;
  // slice 0 straight to stage 0, slices 1 and 2 into register buffers 1 and
  // 0 right behind it; then wait for slice 0 only (its 16 loads went first)
  {
    const SliceRef p0 = lp.template at<MASK>(0), q0 = lq.template at<MASK>(0);
#pragma unroll
    for (int i = 0; i < UPW; ++i) lp.template direct<MASK>(sp, p0, wave, lane, i);
#pragma unroll
    for (int i = 0; i < UPW; ++i) lq.template direct<MASK>(sq, q0, wave, lane, i);
    const int k1 = MASK || klast >= 1 ? 1 : klast, k2 = MASK || klast >= 2 ? 2 : klast;
    const SliceRef p1 = lp.template at<MASK>((int64_t)k1 * BK);
    const SliceRef q1 = lq.template at<MASK>((int64_t)k1 * BK);
#pragma unroll
    for (int i = 0; i < UPW; ++i) S.R[1][i] = lp.template get<MASK>(p1, i);
#pragma unroll
    for (int i = 0; i < UPW; ++i) S.R[1][UPW + i] = lq.template get<MASK>(q1, i);
    const SliceRef p2 = lp.template at<MASK>((int64_t)k2 * BK);
    const SliceRef q2 = lq.template at<MASK>((int64_t)k2 * BK);
#pragma unroll
    for (int i = 0; i < UPW; ++i) S.R[0][i] = lp.template get<MASK>(p2, i);
#pragma unroll
    for (int i = 0; i < UPW; ++i) S.R[0][UPW + i] = lq.template get<MASK>(q2, i);
  }
  asm volatile("s_waitcnt vmcnt(32)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int a = 0; a < NA; ++a) S.FA[a] = frag<PD>(sp, wr * WM + 32 * a, 0, lane);
#pragma unroll
  for (int b = 0; b < NB; ++b) S.FB[0][b] = frag<QD>(sq, wc * WN + 32 * b, 0, lane);
  int k = 0;
  if (ZERO) {
    if (nk == 0) {  // K = 0: the sum is empty
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b) S.acc[a][b] = f32x16_t{};
    } else {
      loop_slice<1, PD, QD, MASK, true>(S, lp, lq, sp, sq, 0, klast, wr, wc, lane);
      loop_slice<0, PD, QD, MASK>(S, lp, lq, sp, sq, 1, klast, wr, wc, lane);
      k = 2;
    }
  }
  for (; k < nk; k += 2) {
    loop_slice<1, PD, QD, MASK>(S, lp, lq, sp, sq, k, klast, wr, wc, lane);
    loop_slice<0, PD, QD, MASK>(S, lp, lq, sp, sq, k + 1, klast, wr, wc, lane);
  }
  // drain the loads of the slices past the end (zeros, never used) and let
  // every wave finish with LDS before the epilogue (or the next pair) reuses it
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __syncthreads();
}

template <class Epi, bool PD, bool QD, bool MASK, int NSEG>
__device__ __forceinline__ void gemm_tile(const Segs<NSEG>& G, int64_t K, int bid, int n_ti,
                                          int n_tj, const typename Epi::Params& ep,
                                          uint16_t* smem) {
  uint16_t LDS_AS* const sp = (uint16_t LDS_AS*)smem;  // P stages: sp + s * BM * BK
  uint16_t LDS_AS* const sq = sp + 2 * BM * BK;         // Q stages: sq + s * BN * BK

  int ti, tj;
  tile_of(bid, n_ti, n_tj, &ti, &tj);
  const int64_t i0 = (int64_t)ti * BM, j0 = (int64_t)tj * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: scalar registers
  const int wr = wave / NWC, wc = wave % NWC;

  LoopState S;
  if (NSEG == 1) {
    // the first k-step writes the accumulators
    mainloop<PD, QD, MASK, true>(S, G.p(0), G.q(0), K, i0, j0, wave, lane, wr, wc, sp, sq);
  } else {
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) S.acc[a][b][r] = 0.0f;
    // one copy of the main loop, run once per pair
#pragma nounroll
    for (int s = 0; s < NSEG; ++s)
      mainloop<PD, QD, MASK, false>(S, G.p(s), G.q(s), K, i0, j0, wave, lane, wr, wc, sp, sq);
  }
  // the epilogue's lane index is computed anew after the loop (from a value
  // the compiler cannot hoist), so no per-lane index lives across the loop
  unsigned z = 0;
  asm volatile("" : "+s"(z));
  const int elane = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, z));
  Epi::apply(ep, S.acc, i0, j0, wr, wc, elane, smem);
}

template <class Epi, bool PD, bool QD, bool MASK, int NSEG>
__global__ __launch_bounds__(NT, 1) void gemm_kernel(Segs<NSEG> G, int64_t K, int n_ti,
                                                     int n_tj, typename Epi::Params ep) {
  __shared__ __attribute__((aligned(1024))) uint16_t smem[kSmemElems];
  gemm_tile<Epi, PD, QD, MASK, NSEG>(G, K, blockIdx.x, n_ti, n_tj, ep, smem);
}

template <class Epi, bool PD, bool QD, int NSEG>
hipError_t run_gemm(const Segs<NSEG>& G, int64_t rows, int64_t cols, int64_t K,
                    const typename Epi::Params& ep, hipStream_t stream) {
  const int64_t n_ti = (rows + BM - 1) / BM, n_tj = (cols + BN - 1) / BN;
  const int64_t n = n_ti * n_tj;
  if (n <= 0) return hipSuccess;
  if (n > INT32_MAX / 2) return hipErrorInvalidValue;
  // every operand has k_limit = K
  if (K % (2 * BK) != 0 || K == 0)
    hipLaunchKernelGGL((gemm_kernel<Epi, PD, QD, true, NSEG>), dim3((unsigned)n), dim3(NT), 0,
                       stream, G, K, (int)n_ti, (int)n_tj, ep);
  else
    hipLaunchKernelGGL((gemm_kernel<Epi, PD, QD, false, NSEG>), dim3((unsigned)n), dim3(NT), 0,
                       stream, G, K, (int)n_ti, (int)n_tj, ep);
  return hipGetLastError();
}

template <class Epi, bool PD, bool QD>
hipError_t run_gemm(const Operand& P, const Operand& Q, int64_t rows, int64_t cols, int64_t K,
                    const typename Epi::Params& ep, hipStream_t stream) {
  return run_gemm<Epi, PD, QD, 1>(Segs<1>{{P}, {Q}}, rows, cols, K, ep, stream);
}

}  // namespace

}  // namespace vce
