// The linear layer over microscaled operands, y = act(x W^T + b) + residual: x in
// e4m3 or e2m1, W in e2m1, both with a scale to 32 columns.
//
// Products run on the scaled matrix instruction, 16 x 16 x 128: lane l holds row
// l % 16 of an operand and supplies the scale of its columns 32 (l / 16) .. + 31.  An
// e2m1 lane holds those 32 columns, 16 bytes; an e4m3 lane holds columns
// 16 (l / 16) .. + 15 and 64 more than these, in the order in which the instruction
// pairs them with the other operand's, whatever its format.
//
// That instruction adds the products of eight consecutive columns with fewer bits than
// float32 has: each is cut toward zero at 2^(e - 13), e the largest sum of two elements'
// exponents among the eight (of products that are not 0); the eights' sums are added in
// float32.  Products of e2m1 by e2m1 span too little to lose anything.  An e4m3 x by
// W loses 5e-6 of the results' 2-norm on normally distributed operands, 2e-5 with columns of
// x that differ in size by e^(+-1) (a float64 model of this, compared with every kernel's results
// to float32's rounding).  16-bit results take that: their own rounding is 1.7e-3 and
// 2.1e-4 of them, and each e4m3 element stands for a value that it is up to 2^-4 off from.  For
// float32 results an e4m3 x and W are expanded to bfloat16, which holds every element and
// scale exactly, for the bf16 instruction with its float32 sums (EXACT below), at half
// the rate and with the expansion: 1024 x 4096 x 4096 76 us for 34 at S = 4.
#include "layer_mx_tile.hpp"

namespace flce {

typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int FMT> constexpr int kMxCode = FMT == kMxE4M3 ? 0 : 4;   // the instruction's name for it

// One 16 x 16 block over 128 columns.  x: the lane's 16 (e2m1) or 32 bytes.
template <int FMT> __device__ __forceinline__ f32x4 mx_mma(const u32x4 (&x)[2], uint32_t xs, u32x4 w, uint32_t ws, f32x4 c) {
  const i32x8 a = {(int)x[0][0], (int)x[0][1], (int)x[0][2], (int)x[0][3], (int)x[1][0], (int)x[1][1], (int)x[1][2], (int)x[1][3]};
  const i32x8 b = {(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, kMxCode<FMT>, 4, 0, (int)xs, 0, (int)ws);
}

// Eight of a lane's 32 columns as bfloat16: columns 8 t .. 8 t + 7 of block l / 16.
template <int FMT> __device__ __forceinline__ u32x4 mx_expand(uint32_t lo, uint32_t hi, uint32_t s) {
  float v[8];
  mx_decode8<FMT>(lo, hi, s, v);
  return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}
template <int FMT> __device__ __forceinline__ void mx_expand32(const u32x4 (&x)[2], uint32_t s, u32x4 (&o)[4]) {
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    if constexpr (FMT == kMxE4M3) o[t] = mx_expand<FMT>(x[t / 2][2 * (t & 1)], x[t / 2][2 * (t & 1) + 1], s);
    else o[t] = mx_expand<FMT>(x[0][t], 0u, s);
  }
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------

// K is copied in blocks: 256 columns of e2m1 by e2m1, 128 of e4m3 by e2m1.  LDS rows
// have 128 bytes, W's beside an e4m3 x 64; 16-byte chunk c of row r lies at place
// c ^ (r % 8), or c ^ (r / 2 % 4), so that eight lanes that read one chunk of
// consecutive rows cover the 128 bytes that the LDS serves them at a time.
template <int FMT> struct MxBlock {
  static constexpr int K = FMT == kMxE4M3 ? 128 : 256;
  static constexpr int kSteps = K / 128;
  static constexpr int kXRow = 128, kWRow = K / 2;
};
template <int ROWB> __device__ __forceinline__ constexpr int mx_place(int row, int chunk) {
  return ROWB == 128 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
}

// Copies of 32 S rows of ROWB bytes.  PERM: tile rows hold weight_row's.
template <int S, int ROWB, bool PERM> struct MxCopy {
  static constexpr int kRows = 1024 / ROWB, kChunks = ROWB / 16, kN = 32 * S / kRows / 4;   // instructions a wave
  uint32_t off[kN];
  int chunk[kN];
  const uint8_t* base;
  int wave;
  __device__ __forceinline__ void init(const uint8_t* p, int64_t ld, int rows, int m0, int tid) {
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    base = p + (int64_t)m0 * ld;
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int t = kRows * (4 * q + wave) + lane / kChunks, row = PERM ? weight_row<S, false>(t) : t;
      chunk[q] = 16 * mx_place<ROWB>(t, lane % kChunks);
      off[q] = m0 + row < rows ? (uint32_t)((int64_t)row * ld + chunk[q]) : kOOB;
    }
  }
  __device__ __forceinline__ void issue(int k0, int kext, lds_t* buf) const {   // bytes of a row
    const __amdgpu_buffer_rsrc_t r = make_rsrc(base + k0);
#pragma unroll
    for (int q = 0; q < kN; ++q) dma16(r, buf + (4 * q + wave) * 1024, k0 + chunk[q] < kext ? off[q] : kOOB);
  }
};

// Copies of both operands' scales: dword d (128 columns) of row r at 4 (32 S d + r), W's
// behind x's.
template <int S, int STEPS> struct MxScales {
  static constexpr int kAll = S * STEPS, kN = (kAll + 3) / 4, kRuns = S / 2;   // 64 rows an instruction
  static constexpr int kBytes = 2 * 128 * S * STEPS;
  uint32_t off[kN];
  const uint8_t* base[2];
  int wave;
  static __device__ __forceinline__ constexpr bool second(int i) { return i >= kRuns * STEPS; }
  __device__ __forceinline__ void init(const uint8_t* xs, int N, int n0, const uint8_t* ws, int F, int f0, int64_t ld, int tid) {
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    base[0] = xs + (int64_t)n0 * ld;
    base[1] = ws + (int64_t)f0 * ld;
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int i = 4 * q + wave, j = second(i) ? i - kRuns * STEPS : i, d = j / kRuns, t = 64 * (j % kRuns) + lane;
      const int row = second(i) ? weight_row<S, false>(t) : t;
      const bool in = i < kAll && (second(i) ? f0 + row < F : n0 + row < N);
      off[q] = in ? (uint32_t)(row * ld + 4 * d) : kOOB;
    }
  }
  __device__ __forceinline__ void issue(int k0, int kext, lds_t* buf) const {   // columns
#pragma unroll
    for (int q = 0; q < kN; ++q) {
      const int i = 4 * q + wave;
      if (kAll % 4 != 0 && i >= kAll) continue;
      const int d = (second(i) ? i - kRuns * STEPS : i) / kRuns;
      const __amdgpu_buffer_rsrc_t r = make_rsrc((second(i) ? base[1] : base[0]) + k0 / kMxBlock);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(buf + 256 * i), 4,
                                               k0 + 128 * d < kext ? off[q] : kOOB, 0, 0, 0);
    }
  }
};

template <int S, int FMT> struct MxLds {
  static constexpr int kX = 32 * S * MxBlock<FMT>::kXRow, kW = 32 * S * MxBlock<FMT>::kWRow;
  static constexpr int kS = MxScales<S, MxBlock<FMT>::kSteps>::kBytes;
};

// The epilogue of one lane's run of C features of token n (features f ..), sums z.
template <class T, int C, bool ACT = true>
__device__ __forceinline__ void mx_finish(const MxLinear& a, int64_t n, int f, const float (&bias)[C], float (&z)[C]) {
  const int64_t o = n * a.F + f;
  const int left = a.F - f;
  float r[C];
  if (a.residual) load_some<T, C>((const T*)a.residual + o, left, r);
#pragma unroll
  for (int e = 0; e < C; ++e) {
    z[e] += bias[e];
    if (ACT) z[e] = act_fwd_rt<T>(a.act, z[e]);
    if (a.residual) z[e] += r[e];
  }
  store_some<T, C>((T*)a.y + o, left, z);
}

// One 32 S x 32 S tile of tokens x features a workgroup (times the K parts): tokens are
// the instruction's rows, features its columns in weight_row's order, so a lane holds S
// consecutive features of a token.  Block b + 1 is copied while block b is computed.
// Two (S = 4) or four workgroups a CU hide one another's waits; LDS traffic bounds full launches (8192 x 4096 x 12288
// e2m1: 334 and 448 us), and the copies' latency a launch of few tiles (48 x 2048 x 8192: 8 us).
// SPLIT: the sums go to a.part and mx_join_kernel does the rest.
template <class T, int FMT, int S, bool SPLIT>
__global__ void __launch_bounds__(256, (S == 4 ? 2 : 4)) mx_linear_kernel(MxLinear a) {
  constexpr bool EXACT = sizeof(T) == 4 && FMT == kMxE4M3;
  typedef MxBlock<FMT> B;
  typedef MxLds<S, FMT> Z;
  __shared__ __attribute__((aligned(16))) char x0[Z::kX], x1[Z::kX], w0[Z::kW], w1[Z::kW], s0[Z::kS], s1[Z::kS];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4, c = lane & 15;
  const int tiles = a.TM * a.TN;
  const int part = SPLIT ? blockIdx.x / tiles : 0;
  int tm, tn;
  tile_coords(blockIdx.x - part * tiles, tiles, a.TM, a.TN, tm, tn);
  const int n0 = tm * 32 * S, f0 = tn * 32 * S, k0 = part * a.kc;
  const int kext = min(a.kc, a.Kp - k0);
  constexpr int XB = FMT == kMxE4M3 ? 2 : 1;   // half bytes of an element
  MxCopy<S, B::kXRow, false> cx;
  MxCopy<S, B::kWRow, true> cw;
  MxScales<S, B::kSteps> cs;
  cx.init(a.x + (int64_t)k0 * XB / 2, (int64_t)a.Kp * XB / 2, a.N, n0, tid);
  cw.init(a.W + k0 / 2, a.Kp / 2, a.F, f0, tid);
  cs.init(a.xs + k0 / kMxBlock, a.N, n0, a.Ws + k0 / kMxBlock, a.F, f0, a.Kp / kMxBlock, tid);
  auto issue = [&](int b, char* x, char* w, char* s) {
    cx.issue(b * B::kXRow, kext * XB / 2, (lds_t*)x);
    cw.issue(b * B::kWRow, kext / 2, (lds_t*)w);
    cs.issue(b * B::K, kext, (lds_t*)s);
  };
  f32x4 acc[S][S];
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int rx = wm * 16 * S + c, rw = wn * 16 * S + c;   // the lane's row in block 0 of either operand
  auto step = [&](const char* x, const char* w, const char* s) {
    const lds_t *X = (const lds_t*)x, *W = (const lds_t*)w, *P = (const lds_t*)s;
    typedef __attribute__((address_space(3))) uint32_t lds_u32;
#pragma unroll
    for (int h = 0; h < B::kSteps; ++h) {
      u32x4 fx[S][2], fw[S][2];
      uint32_t sx[S], sw[S];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int row = rx + 16 * i, ca = FMT == kMxE2M1 ? 4 * h + g : EXACT ? 2 * g : g, cb = EXACT ? 2 * g + 1 : 4 + g;
        fx[i][0] = lds_load16(X + row * B::kXRow + 16 * mx_place<B::kXRow>(row, ca));
        if (FMT == kMxE4M3) fx[i][1] = lds_load16(X + row * B::kXRow + 16 * mx_place<B::kXRow>(row, cb));
        else fx[i][1] = u32x4{0, 0, 0, 0};
        sx[i] = *(const lds_u32*)(P + 4 * (32 * S * h + row)) >> (8 * g);
      }
#pragma unroll
      for (int j = 0; j < S; ++j) {
        const int row = rw + 16 * j;
        fw[j][0] = lds_load16(W + row * B::kWRow + 16 * mx_place<B::kWRow>(row, 4 * h + g));
        fw[j][1] = u32x4{0, 0, 0, 0};
        sw[j] = *(const lds_u32*)(P + Z::kS / 2 + 4 * (32 * S * h + row)) >> (8 * g);
      }
      if constexpr (EXACT) {
        u32x4 ew[S][4];
#pragma unroll
        for (int j = 0; j < S; ++j) mx_expand32<kMxE2M1>(fw[j], sw[j] & 255u, ew[j]);
#pragma unroll
        for (int i = 0; i < S; ++i) {
          u32x4 ex[4];
          mx_expand32<FMT>(fx[i], sx[i] & 255u, ex);
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < S; ++j) mma_frag<uint16_t>(acc[i][j], ex[t], ew[j][t]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j) acc[i][j] = mx_mma<FMT>(fx[i], sx[i], fw[j][0], sw[j], acc[i][j]);
      }
    }
  };
  const int KB = (kext + B::K - 1) / B::K;
  issue(0, x0, w0, s0);
  for (int b = 0; b < KB; b += 2) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (b + 1 < KB) issue(b + 1, x1, w1, s1);
    step(x0, w0, s0);
    if (b + 1 >= KB) break;
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (b + 2 < KB) issue(b + 2, x0, w0, s0);
    step(x1, w1, s1);
  }
  const int f = f0 + (wn * 16 + c) * S;
  float bias[S] = {};
  if (!SPLIT && a.b) load_some<T, S>((const T*)a.b + f, a.F - f, bias);
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int n = n0 + wm * 16 * S + 16 * i + 4 * g + r;
      if (n >= a.N) continue;
      float z[S];
#pragma unroll
      for (int j = 0; j < S; ++j) z[j] = acc[i][j][r];
      if constexpr (SPLIT) store_some<float, S>(a.part + ((int64_t)part * a.N + n) * a.ldp + f, (int)a.ldp - f, z);
      else mx_finish<T, S>(a, n, f, bias, z);
    }
}

// 256 x 256 tiles, for large products (not for EXACT's types): workgroup w computes tiles w, w + grid, ...  The next
// tile's first copies start before the epilogue, and its stores drain under the next tile.  VEC: every lane's run of 8
// features is whole and aligned (F % 8 == 0).
template <class T, int FMT, bool ACT, bool SPLIT, bool VEC>
__global__ void __launch_bounds__(256, 1) mx_linear_big_kernel(MxLinear a) {
  constexpr int XB = FMT == kMxE4M3 ? 2 : 1, ES = sizeof(T);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1, g = lane >> 4, c = lane & 15;
  const int tiles = a.TM * a.TN, total = tiles * a.parts;
  MX_LDS(L);
  MxCopies<FMT> cp;
  int n0, f0, part;
  auto begin = [&](int t) {
    part = SPLIT ? t / tiles : 0;
    int tm, tn;
    tile_coords(t - part * tiles, tiles, a.TM, a.TN, tm, tn);
    n0 = tm * 256;
    f0 = tn * 256;
    cp.k0 = part * a.kc;
    cp.kext = min(a.kc, a.Kp - cp.k0);
    cp.x.init(a.x + (int64_t)cp.k0 * XB / 2, (int64_t)a.Kp * XB / 2, a.N, n0, tid);
    cp.w.init(a.W + cp.k0 / 2, a.Kp / 2, a.F, f0, tid);
    cp.s.init(a.xs, a.N, n0, a.Ws, a.F, f0, a.Kp / kMxBlock, tid);
    cp.begin(L);
  };
  int t = blockIdx.x;
  begin(t);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());   // the tile's first wait allows for an epilogue's stores
  Acc acc;
  while (true) {
    mx_tile_run<FMT, 32>(acc, cp, L, tid);
    const int n0w = n0 + wm * 128, f = f0 + (wn * 16 + c) * 8, ld = SPLIT ? (int)a.ldp : a.F;
    const int64_t base = ((int64_t)part * a.N + n0w) * ld;
    float bias[8] = {};
    if (!SPLIT && a.b) load_some<T, 8>((const T*)a.b + f, a.F - f, bias);
    __builtin_amdgcn_sched_barrier(0);
    // copies that ran past the last step's columns, and the bias
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());
    t += gridDim.x;
    const bool more = t < total;
    if (more) begin(t);
    acc_drain();
    if constexpr (VEC) {
      // Value (i, r) of a lane is token n0w + 4 g + 16 i + r: the lane's byte offset plus the wave's, at most 128 rows.
      const int lim = f < ld ? a.N - n0w - 4 * g : 0;
      const uint32_t lane0 = (uint32_t)(4 * g * ld + f);
      const __amdgpu_buffer_rsrc_t ry = SPLIT ? make_rsrc(a.part + base) : make_rsrc((const T*)a.y + base);
      const __amdgpu_buffer_rsrc_t rr = make_rsrc((const T*)a.residual + base);
      const bool res = !SPLIT && a.residual != nullptr;
      unrolled<8>([&](auto block) {
        constexpr int i = block.value;
        constexpr int S = SPLIT ? 4 : ES;
        float rs[4][8];
        if (!SPLIT && res) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t o = 16 * i + r < lim ? lane0 * S : kOOB;
            if constexpr (ES == 2) {
              buf_load_vec<T, 8>(rr, o, (16 * i + r) * ld * S, rs[r]);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const f32x4 v = __builtin_bit_cast(
                    f32x4, __builtin_amdgcn_raw_buffer_load_b128(rr, o + 16 * h, (16 * i + r) * ld * S, 0));
#pragma unroll
                for (int e = 0; e < 4; ++e) rs[r][4 * h + e] = v[e];
              }
            }
          }
        }
        f32x4 z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = acc_read4(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            v[e] = z[e][r] + bias[e];
            if (ACT) v[e] = act_fwd_rt<T>(a.act, v[e]);
            if (!SPLIT && res) v[e] += rs[r][e];
          }
          const uint32_t o = 16 * i + r < lim ? lane0 * S : kOOB;
          if constexpr (SPLIT) buf_store_vec<float, 8>(ry, o, (16 * i + r) * ld * S, v);
          else buf_store_vec<T, 8>(ry, o, (16 * i + r) * ld * S, v);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
    } else {
      unrolled<8>([&](auto block) {
        constexpr int i = block.value;
        f32x4 z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = acc_read4(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int n = n0w + 16 * i + 4 * g + r;
          if (n >= a.N) continue;
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = z[j][r];
          mx_finish<T, 8, ACT>(a, n, f, bias, v);
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      // lanes past the row stored nothing
      __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());
    }
    if (!more) break;
  }
}

// The epilogue of a split product: thread i takes 8 features of a token.
template <class T> __global__ void __launch_bounds__(256) mx_join_kernel(MxLinear a) {
  const int F8 = (a.F + 7) / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)a.N * F8; i += (int64_t)gridDim.x * 256) {
    const int64_t n = i / F8;
    const int f = (int)(i - n * F8) * 8;
    float z[8] = {}, bias[8] = {};
    for (int p = 0; p < a.parts; ++p) {
      float v[8];
      load_vec<float, 8>(a.part + ((int64_t)p * a.N + n) * a.ldp + f, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] += v[e];
    }
    if (a.b) load_some<T, 8>((const T*)a.b + f, a.F - f, bias);
    mx_finish<T, 8>(a, n, f, bias, z);
  }
}

// ---------------------------------------------------------------------------
// Few tokens
// ---------------------------------------------------------------------------

// Features 16 q .. + 15 of at most 16 tokens a group of waves, which split K among
// them (a.parts waves a group, 8 waves a workgroup); weights go straight to
// registers, two groups of kU loads in flight.  HBM bounds it where K is long (one token,
// 12288 -> 4096, 27 MB: 10 us), its loads' latency where it is not.
constexpr int kMxWaves = 8;
template <class T, int FMT>
__global__ void __launch_bounds__(64 * kMxWaves) mx_linear_skinny_kernel(MxLinear a) {
  constexpr bool EXACT = sizeof(T) == 4 && FMT == kMxE4M3;
  constexpr int kU = 2, XB = FMT == kMxE4M3 ? 2 : 1;
  __shared__ f32x4 red[kMxWaves][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, rl = lane & 15;
  const int groups = kMxWaves / a.parts, f00 = blockIdx.x * 16 * groups, f0 = f00 + 16 * (wave / a.parts);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  if (f0 < a.F) {
    // Rows past F or N repeat the last one: their sums are not stored.
    const int row = min(rl, a.F - 1 - f0), tok = min(rl, a.N - 1), ldw = a.Kp / 2, ldx = a.Kp * XB / 2, lds = a.Kp / kMxBlock;
    const uint32_t offw = (uint32_t)(row * ldw + 16 * g), offx = (uint32_t)(tok * ldx + (EXACT ? 32 : 16) * g);
    const uint32_t offws = (uint32_t)(row * lds), offxs = (uint32_t)(tok * lds);
    const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.W + (int64_t)f0 * ldw), rx = make_rsrc(a.x);
    const __amdgpu_buffer_rsrc_t rws = make_rsrc(a.Ws + (int64_t)f0 * lds), rxs = make_rsrc(a.xs);
    const int steps = a.Kp / 128, per = (steps + a.parts - 1) / a.parts;
    const int t0 = (wave % a.parts) * per, t1 = min(steps, t0 + per);
    u32x4 w[2][kU][2], x[2][kU][2];
    uint32_t ws[2][kU], xs[2][kU];
    auto load = [&](int h, int t) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const bool in = t + u < t1;
        w[h][u][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, in ? offw : kOOB, 64 * (t + u), 0));
        w[h][u][1] = u32x4{0, 0, 0, 0};
        x[h][u][0] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, in ? offx : kOOB, 64 * XB * (t + u), 0));
        if (FMT == kMxE4M3)
          x[h][u][1] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                     rx, in ? offx + (EXACT ? 16 : 64) : kOOB, 64 * XB * (t + u), 0));
        else x[h][u][1] = u32x4{0, 0, 0, 0};
        ws[h][u] = __builtin_amdgcn_raw_buffer_load_b32(rws, in ? offws : kOOB, 4 * (t + u), 0) >> (8 * g);
        xs[h][u] = __builtin_amdgcn_raw_buffer_load_b32(rxs, in ? offxs : kOOB, 4 * (t + u), 0) >> (8 * g);
      }
    };
    auto mma = [&](int h) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if constexpr (EXACT) {
          u32x4 ew[4], ex[4];
          mx_expand32<kMxE2M1>(w[h][u], ws[h][u] & 255u, ew);
          mx_expand32<FMT>(x[h][u], xs[h][u] & 255u, ex);
#pragma unroll
          for (int t = 0; t < 4; ++t) mma_frag<uint16_t>(acc, ew[t], ex[t]);
        } else {
          // W's rows first here: the instruction's operands change places
          const i32x8 wa = {(int)w[h][u][0][0], (int)w[h][u][0][1], (int)w[h][u][0][2], (int)w[h][u][0][3], 0, 0, 0, 0};
          const u32x4 p = x[h][u][0], q = x[h][u][1];
          const i32x8 xb = {(int)p[0], (int)p[1], (int)p[2], (int)p[3], (int)q[0], (int)q[1], (int)q[2], (int)q[3]};
          acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, acc, 4, kMxCode<FMT>, 0, (int)ws[h][u], 0,
                                                                 (int)xs[h][u]);
        }
      }
    };
    load(0, t0);
    for (int t = t0; t < t1; t += 2 * kU) {
      load(1, t + kU);
      mma(0);
      load(0, t + 2 * kU);
      mma(1);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  // Element (token n, feature f) of a group sits in lane 16 (f / 4) + n, value f % 4.
  for (int o = tid; o < groups * 256; o += 64 * kMxWaves) {
    const int q = o >> 8, n = (o >> 4) & 15, fl = o & 15, f = f00 + 16 * q + fl;
    if (n >= a.N || f >= a.F) continue;
    float z[1] = {0.f}, bias[1] = {0.f};
    for (int p = 0; p < a.parts; ++p) z[0] += ((const float*)&red[q * a.parts + p][16 * (fl >> 2) + n])[fl & 3];
    if (a.b) bias[0] = load1<T>((const T*)a.b + f);
    mx_finish<T, 1>(a, n, f, bias, z);
  }
}

// The same for many features: a wave has 64 of them, four blocks that share the token fragments, and all of K.  Four steps
// of weights are under way while four are computed, and their scales come 16 bytes a row at a time.  K >= 512.
// One token, 4096 -> 128256: 62 us (4.5 TB/s of codes and scales); 81 with one block of features a wave, whose loads of x
// and of scales outnumber those of weights four to one.
template <class T, int FMT>
__global__ void __launch_bounds__(256) mx_linear_wide_kernel(MxLinear a) {
  constexpr int XB = FMT == kMxE4M3 ? 2 : 1, G = 4, U = 4;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, rl = lane & 15, f0 = (blockIdx.x * 4 + wave) * 16 * G;
  if (f0 >= a.F) return;
  const int tok = min(rl, a.N - 1), ldw = a.Kp / 2, ldx = a.Kp * XB / 2, lds = a.Kp / kMxBlock, steps = a.Kp / 128;
  const uint32_t offx = (uint32_t)(tok * ldx + 16 * g), offxs = (uint32_t)(tok * lds);
  uint32_t offw[G], offs[G];
#pragma unroll
  for (int q = 0; q < G; ++q) {   // rows past F repeat the last one: their sums are not stored
    const int row = min(16 * q + rl, a.F - 1 - f0);
    offw[q] = (uint32_t)(row * ldw + 16 * g);
    offs[q] = (uint32_t)(row * lds);
  }
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(a.W + (int64_t)f0 * ldw), rx = make_rsrc(a.x);
  const __amdgpu_buffer_rsrc_t rws = make_rsrc(a.Ws + (int64_t)f0 * lds), rxs = make_rsrc(a.xs);
  f32x4 acc[G] = {};
  struct Run {
    u32x4 w[U][G], x[U][XB], ws[G], xs;
  } P, Q;
  auto load16 = [](__amdgpu_buffer_rsrc_t r, uint32_t off, int so) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, so, 0));
  };
  auto load = [&](Run& r, int t) {
    const int run = min(4 * t, lds - 16);   // the last run of a row ends with it
    // the steps of a row one after the other: two share a line
#pragma unroll
    for (int q = 0; q < G; ++q)
#pragma unroll
      for (int u = 0; u < U; ++u) r.w[u][q] = load16(rw, t + u < steps ? offw[q] : kOOB, 64 * (t + u));
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int h = 0; h < XB; ++h) r.x[u][h] = load16(rx, t + u < steps ? offx + 64 * h : kOOB, 64 * XB * (t + u));
#pragma unroll
    for (int q = 0; q < G; ++q) r.ws[q] = load16(rws, t < steps ? offs[q] : kOOB, run);
    r.xs = load16(rxs, t < steps ? offxs : kOOB, run);
  };
  auto mma = [&](Run& r, int t) {
    // dword u + d of a run is step t + u's; steps past K have zeros and a scale of 0
    const int d = t - min(4 * t, lds - 16) / 4;
    auto scale = [&](const u32x4& v, int u) {
      const int i = u + d;
      const uint32_t s = i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3];
      return __builtin_amdgcn_ubfe(s, 8 * g, t + u < steps ? 8 : 0);
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t xs = scale(r.xs, u);
      const u32x4 p = r.x[u][0], p2 = r.x[u][XB - 1];
      const i32x8 xb = {(int)p[0], (int)p[1], (int)p[2], (int)p[3], (int)p2[0], (int)p2[1], (int)p2[2], (int)p2[3]};
#pragma unroll
      for (int q = 0; q < G; ++q) {
        const u32x4 v = r.w[u][q];
        const i32x8 wa = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        acc[q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, acc[q], 4, kMxCode<FMT>, 0, (int)scale(r.ws[q], u), 0,
                                                                  (int)xs);
      }
    }
  };
  // Waves start at different runs of K, and so at different channels of the memory.
  const int runs = (steps + U - 1) / U, first = (blockIdx.x * 4 + wave) % runs;
  auto place = [&](int i) { return U * (i + first < runs ? i + first : i < runs ? i + first - runs : runs); };
  load(P, place(0));
  for (int i = 0; i < runs; i += 2) {
    load(Q, place(i + 1));
    mma(P, place(i));
    load(P, place(i + 2));
    if (i + 1 < runs) mma(Q, place(i + 1));
  }
  // Element (feature 4 g + r, token rl) of a block.
  if (rl >= a.N) return;
#pragma unroll
  for (int q = 0; q < G; ++q) {
    const int f = f0 + 16 * q + 4 * g;
    if (f >= a.F) continue;
    float z[4], bias[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = acc[q][e];
    if (a.b) load_some<T, 4>((const T*)a.b + f, a.F - f, bias);
    mx_finish<T, 4>(a, rl, f, bias, z);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

template <class T, int FMT> static void mx_launch(const MxLinear& a, hipStream_t st) {
  if constexpr (sizeof(T) == 2 || FMT == kMxE2M1) {
    if (a.tile == 1) {
      FLCE_LAUNCH((mx_linear_wide_kernel<T, FMT>), dim3((a.F + 255) / 256), dim3(256), 0, st, a);
      return;
    }
  }
  if (a.tile == 0) {
    const int per = 16 * (kMxWaves / a.parts);
    FLCE_LAUNCH((mx_linear_skinny_kernel<T, FMT>), dim3((a.F + per - 1) / per), dim3(64 * kMxWaves), 0, st, a);
    return;
  }
  const dim3 grid(a.TM * a.TN * a.parts), blk(256);
  if constexpr (sizeof(T) == 2 || FMT == kMxE2M1) {
    if (a.tile == 8) {
      const dim3 persist(grid.x < kPersistGrid ? grid.x : kPersistGrid);
      if (a.parts > 1) FLCE_LAUNCH((mx_linear_big_kernel<T, FMT, false, true, true>), persist, blk, 0, st, a);
      else if (a.F % 8 != 0) FLCE_LAUNCH((mx_linear_big_kernel<T, FMT, true, false, false>), persist, blk, 0, st, a);
      else if (a.act == kActNone) FLCE_LAUNCH((mx_linear_big_kernel<T, FMT, false, false, true>), persist, blk, 0, st, a);
      else FLCE_LAUNCH((mx_linear_big_kernel<T, FMT, true, false, true>), persist, blk, 0, st, a);
    }
  }
  auto tiles = [&](auto s) {
    if (a.parts > 1) FLCE_LAUNCH((mx_linear_kernel<T, FMT, s.value, true>), grid, blk, 0, st, a);
    else FLCE_LAUNCH((mx_linear_kernel<T, FMT, s.value, false>), grid, blk, 0, st, a);
  };
  if (a.tile == 4) tiles(std::integral_constant<int, 4>{});
  else if (a.tile == 2) tiles(std::integral_constant<int, 2>{});
  if (a.parts > 1) {
    const int64_t blocks = ((int64_t)a.N * ((a.F + 7) / 8) + 255) / 256;
    FLCE_LAUNCH((mx_join_kernel<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, a);
  }
}

template <class T> static hipError_t mx_launch_t(const MxLinear& a, hipStream_t st) {
  if (a.format == kMxE4M3) mx_launch<T, kMxE4M3>(a, st);
  else mx_launch<T, kMxE2M1>(a, st);
  return hipGetLastError();
}

hipError_t launch_mx_linear(const MxLinear& a, int dtype, hipStream_t st) {
  return dtype == 1 ? mx_launch_t<uint16_t>(a, st) : dtype == 2 ? mx_launch_t<_Float16>(a, st) : mx_launch_t<float>(a, st);
}

}  // namespace flce
