// Device pieces of the feed-forward operators (the linear layer and the gated
// product): activations with their derivatives, and the operand copies for
// the tile routine of flce_device.hpp that take rows from two weights.
#pragma once

#include <type_traits>

#include "flce_device.hpp"
#include "flce_launch.hpp"

namespace flce {

// ---------------------------------------------------------------------------
// Activations.  T is the tensors' type: 16-bit results need no more than the
// hardware's exp2 and reciprocal (relative error near 2^-22); fp32 results
// take the library's functions.
// ---------------------------------------------------------------------------

template <class T> __device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 4) return 1.f / (1.f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.f + fast_exp2(-kLog2e * z));
}

// Phi(z), the normal distribution function, without branches (the tile
// epilogue holds 256 accumulators, and calls or branches there cost it its
// registers): erfc(x) = t P(t) exp(-x^2) with t = 1 / (1 + p x) for
// x = |z| / sqrt(2) >= 0.  P was fitted to erfc(x) exp(x^2) / t on [0, 9.5] by
// linear programming for the least largest relative error: degree 5 (p = 0.65)
// has 8.7e-6, a 50th of a half step of bf16 or fp16; degree 8 (p = 0.4)
// evaluates to within 3.8e-7 in fp32.  The negative tail keeps that relative
// error, as it takes erfc itself.
template <class T> __device__ __forceinline__ float normal_cdf(float z) {
  const float x = 0.70710678f * fabsf(z);
  const float e = fast_exp2(-0.5f * kLog2e * z * z);
  float t, q;
  if constexpr (sizeof(T) == 4) {
    t = 1.f / fmaf(0.4f, x, 1.f);
    q = 0.04112248122692108f;
    q = fmaf(q, t, -0.1399553418159485f);
    q = fmaf(q, t, 0.0837322324514389f);
    q = fmaf(q, t, 0.08779247105121613f);
    q = fmaf(q, t, 0.08009815216064453f);
    q = fmaf(q, t, 0.19320377707481384f);
    q = fmaf(q, t, 0.2019328773021698f);
    q = fmaf(q, t, 0.22643917798995972f);
    q = fmaf(q, t, 0.22563421726226807f);
  } else {
    t = __builtin_amdgcn_rcpf(fmaf(0.65f, x, 1.f));
    q = 0.144245907664299f;
    q = fmaf(q, t, -0.47328993678092957f);
    q = fmaf(q, t, 0.3572549521923065f);
    q = fmaf(q, t, 0.23146380484104156f);
    q = fmaf(q, t, 0.37395307421684265f);
    q = fmaf(q, t, 0.36638060212135315f);
  }
  const float c = 0.5f * q * t * e;   // Phi(-|z|)
  return z < 0.f ? c : 1.f - c;
}

// 2 k (z + 0.044715 z^3), k = sqrt(2 / pi): gelu's tanh form is z sigmoid of
// it, as (1 + tanh(y)) / 2 = sigmoid(2 y).  z is held to +-20, where the
// sigmoid is already 0 or 1, so that no power of z overflows; a NaN stays.
constexpr float kGelu2k = 1.5957691f;
__device__ __forceinline__ float gelu_clamp(float z) { return z > 20.f ? 20.f : (z < -20.f ? -20.f : z); }
__device__ __forceinline__ float gelu_arg(float zc) { return kGelu2k * zc * (1.f + 0.044715f * zc * zc); }

template <class T, int ACT> __device__ __forceinline__ float act_fwd(float z) {
  if constexpr (ACT == kActRelu) return z < 0.f ? 0.f : z;
  else if constexpr (ACT == kActGelu) return z * normal_cdf<T>(z);
  else if constexpr (ACT == kActGeluTanh) return z * sigmoid<T>(gelu_arg(gelu_clamp(z)));
  else if constexpr (ACT == kActSilu) return z * sigmoid<T>(z);
  else if constexpr (ACT == kActSigmoid) return sigmoid<T>(z);
  else return z;
}

// act(z) into v, and dy * act'(z) returned.  ReLU passes dy where z > 0 (a
// select, so an infinite dy is no NaN elsewhere).
template <class T, int ACT> __device__ __forceinline__ float act_bwd(float z, float dy, float& v) {
  if constexpr (ACT == kActRelu) {
    v = z < 0.f ? 0.f : z;
    return z <= 0.f ? 0.f : dy;
  } else if constexpr (ACT == kActGelu) {
    const float p = normal_cdf<T>(z);
    v = z * p;
    return dy * (p + z * (0.39894228f * fast_exp2(-0.5f * kLog2e * z * z)));
  } else if constexpr (ACT == kActGeluTanh) {
    const float zc = gelu_clamp(z), s = sigmoid<T>(gelu_arg(zc));
    v = z * s;
    return dy * (s + zc * s * (1.f - s) * kGelu2k * (1.f + 3.f * 0.044715f * zc * zc));
  } else if constexpr (ACT == kActSilu) {
    const float s = sigmoid<T>(z);
    v = z * s;
    return dy * (s + v * (1.f - s));
  } else if constexpr (ACT == kActSigmoid) {
    v = sigmoid<T>(z);
    return dy * (v * (1.f - v));
  } else {
    v = z;
    return dy;
  }
}

// The same with the activation known only at run time (uniform branches), for
// the kernels that memory bounds.
template <class T> __device__ __forceinline__ float act_fwd_rt(int act, float z) {
  switch (act) {
    case kActRelu: return act_fwd<T, kActRelu>(z);
    case kActGelu: return act_fwd<T, kActGelu>(z);
    case kActGeluTanh: return act_fwd<T, kActGeluTanh>(z);
    case kActSilu: return act_fwd<T, kActSilu>(z);
    case kActSigmoid: return act_fwd<T, kActSigmoid>(z);
    default: return z;
  }
}

// ---------------------------------------------------------------------------
// Element access
// ---------------------------------------------------------------------------

template <class T> __device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 4) return *(const float*)p;
  else return h16_to_f32<T>(*(const uint16_t*)p);
}
template <class T> __device__ __forceinline__ void store1(T* p, float v) {
  if constexpr (sizeof(T) == 4) *(float*)p = v;
  else *(uint16_t*)p = (uint16_t)(pack2<T>(v, 0.f) & 0xffffu);
}

// C consecutive elements (16-bit: 4 or 8; fp32: 2, 4 or 8) as whole 4- to
// 16-byte accesses from any element's address: rows of odd sizes start on no
// boundary, and global memory takes wide accesses there.
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef f32x2 f32x2_any __attribute__((aligned(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <class T, int C> __device__ __forceinline__ void load_vec(const T* p, float (&v)[C]) {
  if constexpr (sizeof(T) == 4 && C == 2) {
    const f32x2 t = *(const f32x2_any*)p;
    v[0] = t[0];
    v[1] = t[1];
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < C; e += 4) {
      const f32x4 t = *(const f32x4_any*)((const float*)p + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[e + k] = t[k];
    }
  } else {
    uint32_t w[C / 2];
    if constexpr (C == 8) {
      const u32x4 t = *(const u32x4_any*)p;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = t[k];
    } else {
      const u32x2 t = *(const u32x2_any*)p;
      w[0] = t[0];
      w[1] = t[1];
    }
#pragma unroll
    for (int k = 0; k < C / 2; ++k) {
      v[2 * k] = h16_to_f32<T>(w[k]);
      v[2 * k + 1] = h16_to_f32<T>(w[k] >> 16);
    }
  }
}
template <class T, int C> __device__ __forceinline__ void store_vec(T* p, const float (&v)[C]) {
  if constexpr (sizeof(T) == 4 && C == 2) {
    *(f32x2_any*)p = f32x2{v[0], v[1]};
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < C; e += 4) *(f32x4_any*)((float*)p + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
  } else if constexpr (C == 8) {
    *(u32x4_any*)p = u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])};
  } else {
    *(u32x2_any*)p = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
  }
}

// The first `left` of them (any left; none when it is not positive), zeros for the rest.
template <class T, int C> __device__ __forceinline__ void load_some(const T* p, int left, float (&v)[C]) {
  if (left >= C) {
    load_vec<T, C>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e) v[e] = e < left ? load1<T>(p + e) : 0.f;
  }
}
template <class T, int C> __device__ __forceinline__ void store_some(T* p, int left, const float (&v)[C]) {
  if (left >= C) {
    store_vec<T, C>(p, v);
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e)
      if (e < left) store1<T>(p + e, v[e]);
  }
}

// Whole aligned runs through a buffer descriptor: byte offset off (a lane's,
// kOOB reads zeros and stores nothing) plus so (the wave's).
template <class T, int C>
__device__ __forceinline__ void buf_store_vec(__amdgpu_buffer_rsrc_t r, uint32_t off, int so, const float (&v)[C]) {
  if constexpr (sizeof(T) == 4 && C == 2) {
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, f32x2{v[0], v[1]}), r, off, so, 0);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < C; e += 4)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]}), r,
                                             off + 4 * e, so, 0);
  } else if constexpr (C == 8) {
    __builtin_amdgcn_raw_buffer_store_b128(
        u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])}, r, off, so, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])}, r, off, so, 0);
  }
}
template <class T, int C>
__device__ __forceinline__ void buf_load_vec(__amdgpu_buffer_rsrc_t r, uint32_t off, int so, float (&v)[C]) {
  if constexpr (sizeof(T) == 4) {
    static_assert(C == 4 || C == 8, "whole 16-byte pieces");
#pragma unroll
    for (int e = 0; e < C; e += 4) {
      const f32x4 t = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * e, so, 0));
#pragma unroll
      for (int k = 0; k < 4; ++k) v[e + k] = t[k];
    }
  } else {
    static_assert(C == 8, "whole 16-byte pieces");
    const u32x4 t = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, so, 0));
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = h16_to_f32<T>(t[k]);
      v[2 * k + 1] = h16_to_f32<T>(t[k] >> 16);
    }
  }
}

// ---------------------------------------------------------------------------
// Operands over two weights
// ---------------------------------------------------------------------------

// Output tiles, four waves in a 2 x 2 grid of MI x NJ blocks of 16 x 16 each:
// 256 x 256 for 16-bit operands; 128 x 128 for fp32, whose matrix instruction
// is 16 times slower per byte, so that small tiles starve on nothing and two
// workgroups share a CU (one's epilogue runs under the other's products).
template <class T> struct Tile {
  static constexpr int MI = sizeof(T) == 2 ? 8 : 4, NJ = MI;
  static constexpr int M = 32 * MI, N = 32 * NJ;
  static constexpr int kPerCu = sizeof(T) == 2 ? 1 : 2;   // workgroups that fit on a CU
};

// Column order of a tile: in each wave's half (16 NJ rows of the weight
// operand), row 16 j + c (output column c of block j) holds weight row
// NJ c + j, so a lane's NJ blocks of one output row are NJ consecutive columns.
// Gated: the half holds 8 NJ rows of Wg (blocks j < NJ / 2) and the same of Wu:
// row NJ / 2 c + j % (NJ / 2), so a lane has NJ / 2 consecutive columns of g and
// the same of u, and the product act(g) u needs no other lane.
template <int NJ, bool GLU> __device__ __forceinline__ constexpr int weight_row(int t) {
  const int half = t / (16 * NJ), j = t / 16 % NJ, c = t % 16;
  return GLU ? half * 8 * NJ + NJ / 2 * c + j % (NJ / 2) : half * 16 * NJ + NJ * c + j;
}

// 16-bit copies.  Tile row t = 32 q + 8 wave + lane / 8 lies in block
// j = t / 16 % 8 = (2 q + wave / 2) % 8: bit 1 of q alone says which weight.
struct DmaGlu {
  struct Pair {
    __amdgpu_buffer_rsrc_t g, u;
  };
  uint32_t off[8];
  const uint16_t* base[2];
  int wave;
  template <class E>
  __device__ __forceinline__ void init(const E* Wg, const E* Wu, int64_t ld, int F, int f0, int tid) {
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    base[0] = (const uint16_t*)Wg + (int64_t)f0 * ld;
    base[1] = (const uint16_t*)Wu + (int64_t)f0 * ld;
    const int c = (lane & 7) ^ (lane >> 3);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = weight_row<8, true>(8 * (4 * q + wave) + (lane >> 3));
      off[q] = (f0 + row < F) ? (uint32_t)(((int64_t)row * ld + 8 * c) * 2) : kOOB;
    }
  }
  __device__ __forceinline__ Pair rsrc(int k0) const { return {make_rsrc(base[0] + k0), make_rsrc(base[1] + k0)}; }
  template <bool TAIL>
  __device__ __forceinline__ void issue(const Pair& rs, int kleft, lds_t* buf, int lane, int q) const {
    const int c = (lane & 7) ^ (lane >> 3);
    dma16((q & 2) ? rs.u : rs.g, buf + (4 * q + wave) * 1024, (!TAIL || 8 * c < kleft) ? off[q] : kOOB);
  }
};

// Where the input-gradient product reads W: K runs over the rows of Wg and
// then of Wu, each padded to segk (a multiple of the 64-deep copy block, so a
// block lies in one weight), starting at row kbase.  A block's descriptor
// ends with its weight, so rows past F read zeros.  One weight: segk is past
// every K.
struct SegRows {
  const void* p[2];
  int64_t ld;
  int rows, segk, kbase;
  template <int ES>
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int k0, int m0) const {
    const int k = k0 + kbase;
    const bool second = k >= segk;
    const int kk = second ? k - segk : k;
    const char* base = (const char*)(second ? p[1] : p[0]) + ((int64_t)kk * ld + m0) * ES;
    int64_t n = ((int64_t)(rows - kk) * ld - m0) * ES;
    n = n < 0 ? 0 : (n > 0x7fffffff ? 0x7fffffff : n);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, (int)n, 0x00020000);
  }
};

struct DmaSeg {
  Dma<false> d;
  SegRows s;
  int m0;
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int k0) const { return s.rsrc<2>(k0, m0); }
  template <bool TAIL>
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t rs, int kleft, lds_t* buf, int lane, int q) const {
    d.issue<TAIL>(rs, kleft, buf, lane, q);
  }
};

// ---------------------------------------------------------------------------
// fp32 tile: 128 x 128, 32-deep stages through registers into two padded LDS
// buffers per operand, v_mfma_f32_16x16x4_f32.  MFMA bounds it (32 cycles an
// instruction against one 16-byte LDS read per 8 of them).
// ---------------------------------------------------------------------------

constexpr int kF32Rows = 128, kF32K = 32;

// K-contiguous operand of up to two weights: thread (kc, rr) = (tid % 8,
// tid / 8) loads 16 bytes of K of tile rows rr + 32 q.  A gated tile's rows
// 32 q .. 32 q + 31 lie in blocks j = 2 q and 2 q + 1 (mod 4): bit 0 of q tells
// the weight.
template <bool PERM, bool GLU> struct RowStager {
  u32x4 r[4];
  uint32_t off[4];
  const float* base[2];
  int kc4;
  __device__ __forceinline__ void init(const float* p0, const float* p1, int64_t ld, int rows, int m0, int tid) {
    const int rr = tid >> 3;
    kc4 = (tid & 7) * 4;
    base[0] = p0 + (int64_t)m0 * ld;
    base[1] = GLU ? p1 + (int64_t)m0 * ld : base[0];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int t = rr + 32 * q, row = PERM ? weight_row<4, GLU>(t) : t;
      off[q] = m0 + row < rows ? (uint32_t)(((int64_t)row * ld + kc4) * 4) : kOOB;
    }
  }
  __device__ __forceinline__ void load(int k0, int kext) {
    const __amdgpu_buffer_rsrc_t r0 = make_rsrc(base[0] + k0), r1 = make_rsrc(base[1] + k0);
    const bool in = k0 + kc4 < kext;
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = buf_load16(GLU && (q & 1) ? r1 : r0, in ? off[q] : kOOB);
  }
  __device__ __forceinline__ void store(lds_t* buf, int tid) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) lds_store16(buf + ((tid >> 3) + 32 * q) * kRowBytes + (tid & 7) * 16, r[q]);
  }
};

// M-contiguous operand: 4 x 4 blocks transposed in registers, thread (kc, mc)
// = (tid % 8, tid / 8).  SegRows gives the rows (K).
struct ColStager {
  u32x4 r[4];
  uint32_t off[4];
  SegRows s;
  int m0, krow;
  __device__ __forceinline__ void init(const SegRows& rows, int cols, int m0_, int tid) {
    s = rows;
    m0 = m0_;
    krow = (tid & 7) * 4;
    const int m = (tid >> 3) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e) off[e] = m0 + m < cols ? (uint32_t)(((int64_t)(krow + e) * s.ld + m) * 4) : kOOB;
  }
  __device__ __forceinline__ void load(int k0, int kext) {
    const __amdgpu_buffer_rsrc_t rs = s.rsrc<4>(k0, m0);
    const int left = kext - k0 - krow;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = buf_load16(rs, e < left ? off[e] : kOOB);
  }
  __device__ __forceinline__ void store(lds_t* buf, int tid) const {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      lds_store16(buf + ((tid >> 3) * 4 + i) * kRowBytes + (tid & 7) * 16, u32x4{r[0][i], r[1][i], r[2][i], r[3][i]});
  }
};

typedef f32x4 AccF32[4][4];

// acc = the tile's sums over K.  Lane l's 16 bytes of a row are four
// consecutive k; instruction e takes element e, so K runs permuted, the same
// for both operands.
template <class SA, class SB>
__device__ __forceinline__ void gemm_f32(AccF32& acc, SA& sa, int ka, SB& sb, int kb, int K, int tid) {
  __shared__ __attribute__((aligned(16))) char lds[2][2][kF32Rows * kRowBytes];
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int frag = (lane & 15) * kRowBytes + (lane >> 4) * 16;
  const int pa = (wave >> 1) * 64 * kRowBytes + frag, pb = (wave & 1) * 64 * kRowBytes + frag;
  const int KT = (K + kF32K - 1) / kF32K;
  sa.load(0, ka);
  sb.load(0, kb);
  sa.store((lds_t*)lds[0][0], tid);
  sb.store((lds_t*)lds[0][1], tid);
  __syncthreads();
  for (int kt = 0; kt < KT; ++kt) {
    const int cur = kt & 1;
    if (kt + 1 < KT) {
      sa.load((kt + 1) * kF32K, ka);
      sb.load((kt + 1) * kF32K, kb);
    }
    const lds_t* A = (const lds_t*)lds[cur][0];
    const lds_t* B = (const lds_t*)lds[cur][1];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4 a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __builtin_bit_cast(f32x4, lds_load16(A + pa + 16 * i * kRowBytes + 64 * h));
        b[i] = __builtin_bit_cast(f32x4, lds_load16(B + pb + 16 * i * kRowBytes + 64 * h));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i][e], b[j][e], acc[i][j], 0, 0, 0);
    }
    if (kt + 1 < KT) {
      sa.store((lds_t*)lds[cur ^ 1][0], tid);
      sb.store((lds_t*)lds[cur ^ 1][1], tid);
    }
    __syncthreads();
  }
}

// f(integral_constant<int, 0>) .. f(integral_constant<int, N - 1>): an unrolled
// loop whatever its length (the compiler gives up on long ones, and then keeps
// the accumulators they index in memory).
template <int N, class F> __device__ __forceinline__ void unrolled(F&& f) {
  if constexpr (N > 0) {
    unrolled<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// One block's sums in vector registers.
template <class T> __device__ __forceinline__ f32x4 block_sums(const f32x4& blk) {
  if constexpr (sizeof(T) == 2) return acc_read4(blk);
  else return blk;
}

}  // namespace flce
