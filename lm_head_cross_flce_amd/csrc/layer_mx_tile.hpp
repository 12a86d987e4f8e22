// The 256 x 256 tile of the microscaled product, on the schedule of flce_device.hpp's tile routine: four waves of
// 128 x 128 each, 8 x 8 blocks of 16 x 16 in accumulation registers; operands go to LDS by the buffer unit; every
// instruction has its slot.
//
// A step is the instruction's 128 columns, 1024 cycles of it with e2m1 operands (four times the rate of bfloat16) and
// 2048 with an e4m3 x.  What feeds it has to come in whole 128-byte lines: 128 bytes of a row at a time, 256 columns of
// e2m1 or 128 of e4m3, and scales for four steps, 16 bytes of a row.  (64 bytes of an e2m1 row and a dword of its scales
// a step through four buffers, copies three steps ahead: 281 us for 8192 x 4096 x 12288, 203 so, on one box.)
//
// 8192 x 4096 x 12288: e2m1 206 us (4.0 PFLOP/s), e4m3 293 (2.8); 4096 x 8192 x 8192: 124 and 178; boxes differ by 3%.
// The matrix instructions are busy for 50% of the active cycles with e2m1 operands and for 67% with an e4m3 x, at the
// 1.9 to 2.0 GHz that the power limit leaves.  The waves' cycles are 18% and 11% at waits and 24% and 49% for an
// instruction to issue; LDS serves reads in 25% and 21% of the cycles, a quarter and a fifth of that bank conflicts.
#pragma once

#include "layer_mx_device.hpp"

namespace flce {

// x's and W's elements for the instruction (0: e4m3, 4: e2m1); the accumulator is tied to the destination as in
// mfma16, and acc_drain() must precede any read of it.  The matrix instruction needs two wait states after a vector
// instruction that wrote one of its operands, which the compiler does not see to for inline assembly.  Here only the
// scales are such, and mx_stage sets them at least six slots before their first use; should a compiler put a copy of
// another operand in between, the build fails (matrix_waits.py reads the code that it made).  (Waits in the assembly itself
// would cost a quarter of the e2m1 tile's issue cycles: 238 us for 8192 x 4096 x 12288, for 203 on one box.)
template <int FMT, bool ZERO, class A>
__device__ __forceinline__ void mx_mfma(f32x4& c, const A& a, uint32_t sa, const u32x4& b, uint32_t sb) {
#ifdef __HIP_DEVICE_COMPILE__   // the host's pass has no registers of 32 bytes
  if constexpr (FMT == kMxE4M3) {
    if (ZERO)
      asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0] blgp:4"
                   : "=a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else
      asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] blgp:4"
                   : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  } else {
    if (ZERO)
      asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, 0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                   : "=a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
    else
      asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
                   : "+a"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb));
  }
#endif
}

// Copies of 128 bytes of 256 rows: 16-byte chunk c of row r lies at place c ^ (r % 8), so that eight lanes that read one
// chunk of consecutive rows cover all banks.  PERM: tile rows hold weight_row's.
template <bool PERM> struct MxDma {
  uint32_t off[8];
  const uint8_t* base;
  int wave, c;
  __device__ __forceinline__ void init(const uint8_t* p, int64_t ld, int rows, int m0, int tid) {
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    base = p + (int64_t)m0 * ld;
    c = 16 * ((lane & 7) ^ (lane >> 3));
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int t = 8 * (4 * q + wave) + (lane >> 3), row = PERM ? weight_row<8, false>(t) : t;
      off[q] = m0 + row < rows ? (uint32_t)((int64_t)row * ld + c) : kOOB;
    }
  }
  // k0, left: bytes of a row.  TAIL: the run may reach past the row's end.
  template <bool TAIL> __device__ __forceinline__ void issue(int k0, int left, lds_t* buf, int q) const {
    dma16(make_rsrc(base + k0), buf + (4 * q + wave) * 1024, !TAIL || c < left ? off[q] : kOOB);
  }
};

// Copies of both operands' scales, 16 bytes a row (four steps): x's 256 rows, then W's.  A row's last run starts so that
// it ends with the row (mx_scale_run).
struct MxScaleDma {
  uint32_t off[2];
  const uint8_t* base[2];
  int wave, bytes;   // of a row
  __device__ __forceinline__ void init(const uint8_t* xs, int N, int n0, const uint8_t* ws, int F, int f0, int64_t ld, int tid) {
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    base[0] = xs + (int64_t)n0 * ld;
    base[1] = ws + (int64_t)f0 * ld;
    bytes = (int)ld;
    const int row = weight_row<8, false>(tid);
    off[0] = n0 + tid < N ? (uint32_t)(tid * ld) : kOOB;
    off[1] = f0 + row < F ? (uint32_t)(row * ld) : kOOB;
  }
  __device__ __forceinline__ void issue(int k, lds_t* buf, int q) const {   // k: a column of the whole row
    dma16(make_rsrc(base[q] + mx_scale_run(k, bytes)), buf + 4096 * q + 1024 * wave, off[q]);
  }
};

template <int FMT> struct MxTile {
  static constexpr int kXSteps = FMT == kMxE4M3 ? 1 : 2;   // steps of x's 128 bytes; W's have two
  static constexpr int kCarry = FMT == kMxE4M3 ? 2 : 4;    // rows of blocks that a step leaves to the next
};

struct MxBuf {
  lds_t *x[2], *w[2], *s[2];
};
// Each buffer is its own object, so that the compiler need not wait for copies into one before reads of another.
#define MX_LDS(name)                                                                                                   \
  __shared__ __attribute__((aligned(16))) char name##_x0[32768], name##_x1[32768], name##_w0[32768], name##_w1[32768]; \
  __shared__ __attribute__((aligned(16))) char name##_s0[8192], name##_s1[8192];                                       \
  const MxBuf name {                                                                                                   \
    {(lds_t*)name##_x0, (lds_t*)name##_x1}, {(lds_t*)name##_w0, (lds_t*)name##_w1}, {(lds_t*)name##_s0, (lds_t*)name##_s1} \
  }

template <int FMT> struct MxCopies {
  MxDma<false> x;
  MxDma<true> w;
  MxScaleDma s;
  int k0, kext;   // the part's first column in the whole row (a multiple of 256), its columns (of 128)
  static constexpr int xb(int k) { return FMT == kMxE4M3 ? k : k / 2; }   // bytes of k columns of x
  // One of eight instructions of x's and of W's runs from column k, one of two of the scales'.  Past the part's end x
  // and W read zeros; scales there are not used.
  template <bool TAIL> __device__ __forceinline__ void copy_x(int k, lds_t* buf, int q) const {
    x.template issue<TAIL>(xb(k), xb(kext - k), buf, q);
  }
  template <bool TAIL> __device__ __forceinline__ void copy_w(int k, lds_t* buf, int q) const {
    w.template issue<TAIL>(k / 2, (kext - k) / 2, buf, q);
  }
  __device__ __forceinline__ void copy_s(int k, lds_t* buf, int q) const { s.issue(k0 + k, buf, q); }
  // The first two runs of x and W and the first of the scales; every wave has left the tile before.
  __device__ __forceinline__ void begin(const MxBuf& L) const {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int q = 0; q < 8; ++q) copy_x<true>(128 * MxTile<FMT>::kXSteps * r, L.x[r], q);
#pragma unroll
      for (int q = 0; q < 8; ++q) copy_w<true>(256 * r, L.w[r], q);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) copy_s(0, L.s[0], q);
  }
};

// Per-lane LDS addresses.  h: e2m1, the step of the run; of an e4m3 x, the half of the fragment.
struct MxFrag {
  int x[2], w[2], s[2];
  __device__ __forceinline__ void init(int wm, int wn, int lane) {
    const int r = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[h] = (wm * 128 + r) * 128 + 16 * ((4 * h + g) ^ (r & 7));
      w[h] = (wn * 128 + r) * 128 + 16 * ((4 * h + g) ^ (r & 7));
    }
    s[0] = 16 * (wm * 128 + r);
    s[1] = 16 * (256 + wn * 128 + r);
  }
};

template <int FMT> struct MxRegs {
  typedef uint32_t u32xa __attribute__((ext_vector_type(FMT == kMxE4M3 ? 8 : 4)));
  u32xa a[8];
  u32x4 b[8];
  uint32_t sa[8], sb[8];
};

// Step Q of eight (the scale buffers' two runs), columns k .. k + 127.  First the step before's last kCarry rows of
// blocks, while this step's scales and fragments of W and of x's first four blocks are read, then its own rows
// 0 .. 7 - kCarry, while x's other blocks are.  The first step that reads a run copies the next one into the buffer that
// the run before left, as soon as it can; the last one ends with the wait for those copies and the barrier that publishes
// them and frees this run's buffer.
template <int FMT, int Q, bool FIRST, bool SECOND, bool TAIL>
__device__ __forceinline__ void mx_stage(Acc& acc, MxRegs<FMT>& P, MxRegs<FMT>& C, const MxFrag& f, const MxBuf& L,
                                         const MxCopies<FMT>& cp, int k, int shift) {
  typedef MxTile<FMT> G;
  constexpr int XS = G::kXSteps, RA = 3 - XS;
  constexpr int xi = Q / XS % 2, wi = Q / 2 % 2, si = Q / 4 % 2, xh = XS == 2 ? Q % 2 : 0;
  constexpr bool kCopyX = Q % XS == 0 && !FIRST, kCopyW = Q % 2 == 0 && !FIRST, kCopyS = Q % 4 == 1, kEnd = XS == 1 || Q % 2 == 1;
  // copies that may stay in flight at its end: e4m3, W's of an even step; the scales', but for their last step; all while
  // the tile's first copies are enough (the stores of the tile before are among them)
  constexpr int VMW = FIRST || (SECOND && XS == 2) ? 63 : XS == 1 && Q % 2 == 0 ? 8 : Q % 4 == 1 ? 2 : 0;
  constexpr int kFirst = 8 * G::kCarry;
  static_assert(kFirst == 32 || kFirst == 16, "the plan below");
  const lds_t *bx = L.x[xi], *bw = L.w[wi], *bs = L.s[si];
  typedef __attribute__((address_space(3))) uint32_t lds_u32;
  auto read_a = [&](int i, int h) {
    const u32x4 v = lds_load16(bx + f.x[XS == 2 ? xh : h] + 2048 * i);
#pragma unroll
    for (int e = 0; e < 4; ++e) C.a[i][4 * h + e] = v[e];
  };
  // Copy i of the step's: x's, W's, the scales'.
  auto copy = [&](int i) {
    if (kCopyX && i >= 0 && i < 8) cp.template copy_x<TAIL>(k + 128 * XS, L.x[xi ^ 1], i);
    if (kCopyX) i -= 8;
    if (kCopyW && i >= 0 && i < 8) cp.template copy_w<TAIL>(k + 256, L.w[wi ^ 1], i);
    if (kCopyW) i -= 8;
    if (kCopyS && i >= 0 && i < 2) cp.copy_s(k - 128 + 512, L.s[si ^ 1], i);
  };
  // where this step's dword lies in its run, and whether the part has the step at all (its scales are 0 if not)
  const int at = mx_scale_place(cp.k0 + k, cp.k0 + k - 128 * (Q % 4), cp.s.bytes);
  const uint32_t width = !TAIL || k < cp.kext ? 8 : 0;
  const lds_t *ps = bs + f.s[0] + at, *pw = bs + f.s[1] + at;
  uint32_t raw[16];
#pragma unroll
  for (int k1 = 0; k1 < kFirst; ++k1) {
    constexpr int i0 = 8 - G::kCarry;
    if (!FIRST) mx_mfma<FMT, SECOND>(acc[i0 + k1 / 8][k1 % 8], P.a[i0 + k1 / 8], P.sa[i0 + k1 / 8], P.b[k1 % 8], P.sb[k1 % 8]);
    // the scales, x's 0..7 and W's 8..15: read in the first slots, the lane's columns' byte taken out eight slots later
    constexpr int per = kFirst == 32 ? 1 : 2;
#pragma unroll
    for (int e = per * k1; e < per * (k1 + 1); ++e)
      if (e < 16) raw[e] = *(const lds_u32*)((e < 8 ? ps : pw) + 256 * (e & 7));
#pragma unroll
    for (int e = per * (k1 - 8); e < per * (k1 - 7); ++e)
      if (e >= 0 && e < 16) (e < 8 ? C.sa[e & 7] : C.sb[e & 7]) = __builtin_amdgcn_ubfe(raw[e], shift, width);
    if (k1 < 8) C.b[k1] = lds_load16(bw + f.w[Q % 2] + 2048 * k1);
    else if (k1 < 8 + 4 * RA) read_a((k1 - 8) / RA, (k1 - 8) % RA);
    if (kFirst == 32 ? (k1 & 1) == 0 : true) copy(kFirst == 32 ? k1 / 2 : k1);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int k2 = 0; k2 < 64 - kFirst; ++k2) {
    mx_mfma<FMT, FIRST>(acc[k2 / 8][k2 % 8], C.a[k2 / 8], C.sa[k2 / 8], C.b[k2 % 8], C.sb[k2 % 8]);
    // x's block 4 + i: at once (e2m1), or as row i begins
    if (kFirst == 32 ? k2 < 4 * RA : k2 < 32 && k2 % 8 < RA) {
      if (kFirst == 32) read_a(4 + k2 / RA, k2 % RA);
      else read_a(4 + k2 / 8, k2 % 8);
    }
    if (k2 < 4) copy(16 + k2);
    __builtin_amdgcn_sched_barrier(0);
  }
  if constexpr (kEnd) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<VMW>());
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  }
}

// acc = the tile's sums over cp.kext columns; cp.begin has run, and at least EXTRA memory operations of every wave after
// it, which may stay in flight.  acc_drain() before reading them.
template <int FMT, int EXTRA> __device__ __forceinline__ void mx_tile_run(Acc& acc, const MxCopies<FMT>& cp, const MxBuf& L, int tid) {
  const int lane = tid & 63, wave = tid >> 6, shift = 8 * (lane >> 4);
  MxFrag f;
  f.init(wave >> 1, wave & 1, lane);
  // Steps run in pairs, fragments by turns in X and Y; a step past K has zeros.
  const int pairs = (cp.kext + 255) / 256;
  MxRegs<FMT> X, Y;
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<EXTRA>());
  __builtin_amdgcn_s_barrier();
  int k = 0;
  using std::integral_constant;
  auto pair = [&](auto q, auto first, auto tail) {
    constexpr bool F = first.value, T = tail.value;
    mx_stage<FMT, q.value, F, false, T>(acc, Y, X, f, L, cp, k, shift);
    mx_stage<FMT, q.value + 1, false, F, T>(acc, X, Y, f, L, cp, k + 128, shift);
    k += 256;
  };
  typedef std::true_type Yes;
  typedef std::false_type No;
  pair(integral_constant<int, 0>{}, Yes{}, Yes{});
  int p = 1;
  auto four = [&](auto tail) {
    pair(integral_constant<int, 2>{}, No{}, tail);
    pair(integral_constant<int, 4>{}, No{}, tail);
    pair(integral_constant<int, 6>{}, No{}, tail);
    pair(integral_constant<int, 0>{}, No{}, tail);
    p += 4;
  };
  while (256 * (p + 5) <= cp.kext) four(No{});   // every column that the four pairs use or copy is inside K
  if (p + 4 <= pairs) four(Yes{});
  if (p < pairs) {
    pair(integral_constant<int, 2>{}, No{}, Yes{});
    if (p + 1 < pairs) {
      pair(integral_constant<int, 4>{}, No{}, Yes{});
      if (p + 2 < pairs) pair(integral_constant<int, 6>{}, No{}, Yes{});
    }
  }
#pragma unroll
  for (int q = 0; q < 8 * MxTile<FMT>::kCarry; ++q) {
    constexpr int i0 = 8 - MxTile<FMT>::kCarry;
    mx_mfma<FMT, false>(acc[i0 + q / 8][q % 8], Y.a[i0 + q / 8], Y.sa[i0 + q / 8], Y.b[q % 8], Y.sb[q % 8]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace flce
