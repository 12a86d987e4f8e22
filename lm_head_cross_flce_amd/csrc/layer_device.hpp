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

// exp(-z^2 / 2).  The argument of exp2 is up to 126 in size, and its float32
// rounding would be as large a relative error of the result: 8e-6 at z = -12.  fp32
// keeps it in two floats (z^2 and its product with log2(e) / 2 with their fma
// remainders): 2e-7.  z is held to 16, past which the result is 0, so that no
// remainder is infinity less infinity; the callers' other terms keep a NaN.
template <class T> __device__ __forceinline__ float gauss(float z) {
  constexpr float c = -0.5f * kLog2e;
  if constexpr (sizeof(T) == 4) {
    constexpr float c_lo = (float)(-0.5 * 1.4426950408889634 - (double)c);
    const float a = fminf(fabsf(z), 16.f), s = a * a, hi = c * s;
    const float lo = fmaf(c_lo, s, fmaf(c, fmaf(a, a, -s), fmaf(c, s, -hi)));
    const float e = fast_exp2(hi);
    return fmaf(0.69314718f * e, lo, e);
  } else {
    return fast_exp2(c * z * z);
  }
}

// Phi(z), the normal distribution function, without branches (the tile
// epilogue holds 256 accumulators, and calls or branches there cost it its
// registers): erfc(x) = t P(t) exp(-x^2) with t = 1 / (1 + p x) for
// x = |z| / sqrt(2) >= 0.  P was fitted to erfc(x) exp(x^2) / t on [0, 9.5] by
// linear programming for the least largest relative error: degree 5 (p = 0.65)
// has 8.7e-6, a 50th of a half step of bf16 or fp16; degree 8 (p = 0.4)
// evaluates to within 3.8e-7 in fp32, and with gauss the tail to 4.6e-7 of itself
// down to z = -12.9, as it takes erfc itself.
template <class T> __device__ __forceinline__ float normal_cdf(float z) {
  const float x = 0.70710678f * fabsf(z);
  const float e = gauss<T>(z);
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
    return dy * (p + z * (0.39894228f * gauss<T>(z)));
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

// C consecutive elements (1, 2, 4 or 8) as whole accesses of up to 16 bytes from any element's address: rows of odd sizes start on no
// boundary, and global memory takes wide accesses there.
typedef uint32_t u32_any __attribute__((aligned(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef f32x2 f32x2_any __attribute__((aligned(4)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

template <class T, int C> __device__ __forceinline__ void load_vec(const T* p, float (&v)[C]) {
  if constexpr (C == 1) {
    v[0] = load1<T>(p);
  } else if constexpr (sizeof(T) == 4 && C == 2) {
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
    } else if constexpr (C == 4) {
      const u32x2 t = *(const u32x2_any*)p;
      w[0] = t[0];
      w[1] = t[1];
    } else {
      w[0] = *(const u32_any*)p;
    }
#pragma unroll
    for (int k = 0; k < C / 2; ++k) {
      v[2 * k] = h16_to_f32<T>(w[k]);
      v[2 * k + 1] = h16_to_f32<T>(w[k] >> 16);
    }
  }
}
template <class T, int C> __device__ __forceinline__ void store_vec(T* p, const float (&v)[C]) {
  if constexpr (C == 1) {
    store1<T>(p, v[0]);
  } else if constexpr (sizeof(T) == 4 && C == 2) {
    *(f32x2_any*)p = f32x2{v[0], v[1]};
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < C; e += 4) *(f32x4_any*)((float*)p + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
  } else if constexpr (C == 8) {
    *(u32x4_any*)p = u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])};
  } else if constexpr (C == 4) {
    *(u32x2_any*)p = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
  } else {
    *(u32_any*)p = pack2<T>(v[0], v[1]);
  }
}

__device__ __forceinline__ float buf_load4(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
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

// Whole aligned runs of 4 or 8 elements through a buffer descriptor: byte
// offset off (a lane's, kOOB reads zeros and stores nothing) plus so (the
// wave's).
template <class T, int C>
__device__ __forceinline__ void buf_store_vec(__amdgpu_buffer_rsrc_t r, uint32_t off, int so, const float (&v)[C]) {
  if constexpr (C < 4) {
    // not taken: small tiles store through store_some
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
// Eight 16-bit elements (other C are never taken; the type is for code that is not reached).
template <class T, int C>
__device__ __forceinline__ void buf_load_vec(__amdgpu_buffer_rsrc_t r, uint32_t off, int so, float (&v)[C]) {
  if constexpr (C == 8) {
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

// Output tiles of 32 S x 32 S, four waves in a 2 x 2 grid of S x S blocks of
// 16 x 16 each.  S = 8 (16-bit only) is the tile routine of flce_device.hpp:
// one workgroup a CU, the best rate on large products.  S = 4 and 2 run two and
// four workgroups a CU, so that one's epilogue and first loads run under the
// others' products, and cut small products finely enough to fill the CUs.
template <class T, int S_> struct Tile {
  static_assert(S_ == 2 || S_ == 4 || (S_ == 8 && sizeof(T) == 2), "tile sizes");
  static constexpr int S = S_, M = 32 * S;
  // workgroups a CU should hold; fp32's staged values need a third more registers
  static constexpr int kPerCu = S == 8 ? 1 : S == 4 ? 2 : sizeof(T) == 4 ? 3 : 4;
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
// Small tiles (S = 4, 2): operands of 32 S rows, two LDS buffers each, plain
// loops; the other workgroups of the CU cover the waits.
// ---------------------------------------------------------------------------

// One 16 x 16 block from 16 bytes of K per lane of either operand.  fp32: the
// lane's four consecutive k go to four instructions, so K runs permuted, the
// same for both operands.
template <class T> __device__ __forceinline__ void mma_frag(f32x4& c, const u32x4& a, const u32x4& b) {
  if constexpr (sizeof(T) == 4) {
    const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[e], fb[e], c, 0, 0, 0);
  } else if constexpr (IsF16<T>::value) {
    typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                0);
  }
}

// Whether pass q of a gated weight tile's copies (32 tile rows; the caller's
// wave / 2 takes rows 16 (wave / 2) .. + 15 of them, block 2 q + wave / 2) reads
// Wu.  S = 2: the wave alone decides, so its base is chosen once.
template <int S> __device__ __forceinline__ constexpr bool pass_is_up(int q) { return S > 2 && (2 * q) % S >= S / 2; }

// 16-bit K-contiguous operand, LDS rows of 128 bytes (64 k) with 16-byte chunk
// p of row r holding chunk p ^ (r & 7).
template <class T, int S, bool PERM, bool GLU> struct RowCopy {
  static constexpr int kBytes = 32 * S * 128;
  uint32_t off[S];
  const uint16_t* base[2];
  int wave, c8;
  __device__ __forceinline__ void init(const T* p0, const T* p1, int64_t ld, int rows, int m0, int tid) {
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    c8 = 8 * ((lane & 7) ^ (lane >> 3));
    base[0] = (const uint16_t*)p0 + (int64_t)m0 * ld;
    base[1] = GLU ? (const uint16_t*)p1 + (int64_t)m0 * ld : base[0];
    if (S == 2 && (wave >> 1)) base[0] = base[1];
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int t = 8 * (4 * q + wave) + (lane >> 3), row = PERM ? weight_row<S, GLU>(t) : t;
      off[q] = m0 + row < rows ? (uint32_t)(((int64_t)row * ld + c8) * 2) : kOOB;
    }
  }
  __device__ __forceinline__ void issue(int k0, int kext, lds_t* buf) const {
    const __amdgpu_buffer_rsrc_t r0 = make_rsrc(base[0] + k0), r1 = make_rsrc(base[1] + k0);
    const bool in = k0 + c8 < kext;
#pragma unroll
    for (int q = 0; q < S; ++q) dma16(GLU && pass_is_up<S>(q) ? r1 : r0, buf + (4 * q + wave) * 1024, in ? off[q] : kOOB);
  }
};
template <int S> struct RowFrag {
  int base[2];
  __device__ __forceinline__ void init(int wbase, int lane) {
    const int rl = lane & 15, c = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) base[h] = (wbase + rl) * 128 + 16 * ((4 * h + c) ^ (rl & 7));
  }
  __device__ __forceinline__ u32x4 read(const lds_t* buf, int half, int i) const {
    return lds_load16(buf + base[half] + 2048 * i);
  }
};

// 16-bit M-contiguous operand: LDS rows (one per k) of 64 S bytes, chunk p of
// row k holding chunk p ^ col_swz(k); read with the transposing loads (see
// flce_device.hpp).  The swizzle spreads the eight 32-byte runs that the LDS
// serves in a cycle (four rows of two groups 8 rows apart) over its 256 bytes:
// rows of 128 bytes already alternate halves.
template <int S> __device__ __forceinline__ constexpr int col_swz(int k) {
  return S == 2 ? (2 * ((k >> 1) & 1)) | (4 * ((k >> 3) & 1)) : mswz(k);
}
template <class T, int S> struct ColCopy {
  static constexpr int kBytes = 32 * S * 128;
  uint32_t off[S];
  SegRows s;
  int m0, wave;
  __device__ __forceinline__ void init(const SegRows& rows, int cols, int m0_, int tid) {
    s = rows;
    m0 = m0_;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int k = (4 * q + wave) * (16 / S) + lane / (4 * S), c = (lane % (4 * S)) ^ col_swz<S>(k);
      off[q] = m0 + 8 * c < cols ? (uint32_t)(((int64_t)k * s.ld + 8 * c) * 2) : kOOB;
    }
  }
  __device__ __forceinline__ void issue(int k0, int, lds_t* buf) const {
    const __amdgpu_buffer_rsrc_t rs = s.rsrc<2>(k0, m0);
#pragma unroll
    for (int q = 0; q < S; ++q) dma16(rs, buf + (4 * q + wave) * 1024, off[q]);
  }
};
template <int S> struct ColFrag {
  int a[2][S];
  __device__ __forceinline__ void init(int wbase, int lane) {
    const int j = lane & 15, G = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int k = 8 * G + 4 * h + (j >> 2), m = wbase + 16 * i + 4 * (j & 3);
        a[h][i] = k * 64 * S + 16 * ((m >> 3) ^ col_swz<S>(k)) + 2 * (m & 7);
      }
  }
  __device__ __forceinline__ u32x4 read(const lds_t* buf, int half, int i) const {
    typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4;
    u32x4 f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const u32x2 v = __builtin_bit_cast(
          u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(buf + 2048 * S * half + a[h][i])));
      f[2 * h] = v[0];
      f[2 * h + 1] = v[1];
    }
    return f;
  }
};

// A small tile's LDS buffers, declared by the kernel (SMALL_LDS): 16-bit, two
// an operand; fp32, one (in p[0] and p[2]).
struct SmallLds {
  lds_t* p[4];
};
template <class T, int S> struct SmallLdsSize {
  static constexpr int kA = 32 * S * (sizeof(T) == 2 ? 128 : 208), kB = sizeof(T) == 2 ? kA : 16;
};
#define SMALL_LDS(name, T, S)                                                             \
  __shared__ __attribute__((aligned(16))) char name##_0[SmallLdsSize<T, S>::kA];           \
  __shared__ __attribute__((aligned(16))) char name##_1[SmallLdsSize<T, S>::kB];           \
  __shared__ __attribute__((aligned(16))) char name##_2[SmallLdsSize<T, S>::kA];           \
  __shared__ __attribute__((aligned(16))) char name##_3[SmallLdsSize<T, S>::kB];           \
  const SmallLds name {                                                                   \
    { (lds_t*)name##_0, (lds_t*)name##_1, (lds_t*)name##_2, (lds_t*)name##_3 }            \
  }

// acc = the tile's sums over K, 16-bit.  Block b + 1 is copied while block b is
// computed; the barrier at the head of a block publishes it and frees the other
// buffer.  Each buffer is its own object, so that the compiler need not wait
// for copies into one before reads of the other.  Both stages' fragments are
// read ahead of the products, which run at raised priority: the CU's other
// workgroups fill the waits (4096 x 4096 x 1024 bf16 at S = 4: 40.0 -> 37.6 us).
template <class T, int S, class FA, class FB, class CA, class CB>
__device__ __forceinline__ void gemm_small(f32x4 (&acc)[S][S], const CA& ca, int ka, const CB& cb, int kb, int K,
                                           const SmallLds& L, int tid) {
  lds_t *const a0 = L.p[0], *const a1 = L.p[1], *const b0 = L.p[2], *const b1 = L.p[3];
  const int lane = tid & 63, wave = tid >> 6;
  FA fa;
  FB fb;
  fa.init((wave >> 1) * 16 * S, lane);
  fb.init((wave & 1) * 16 * S, lane);
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int KB = (K + kBlockK - 1) / kBlockK;
  if (KB < 1) return;   // no copy may be under way when the workgroup ends
  ca.issue(0, ka, a0);
  cb.issue(0, kb, b0);
  auto step = [&](int b, const lds_t* A, const lds_t* B, lds_t* nA, lds_t* nB) {
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    if (b + 1 < KB) {
      ca.issue((b + 1) * kBlockK, ka, nA);
      cb.issue((b + 1) * kBlockK, kb, nB);
    }
    u32x4 x[2][S], y[2][S];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < S; ++i) x[h][i] = fa.read(A, h, i);
#pragma unroll
      for (int j = 0; j < S; ++j) y[h][j] = fb.read(B, h, j);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int j = 0; j < S; ++j) mma_frag<T>(acc[i][j], x[h][i], y[h][j]);
    __builtin_amdgcn_s_setprio(0);
  };
  for (int b = 0; b < KB; b += 2) {
    step(b, a0, b0, a1, b1);
    if (b + 1 < KB) step(b + 1, a1, b1, a0, b0);
  }
}

// fp32 products on the bf16 matrix cores.  A float's 24 significant bits are
// exactly three bfloat16 parts of 8, x = h + m + l: h is x rounded to nearest, m and
// l cut off what it leaves, |m| <= 2^-8 |x|, |l| < 2^-15 |x|.  Of the nine products of
// parts the six of weight 2^-16 or more, hh + hm + mh + hl + lh + mm, give x y to 2^-22
// relative and mostly nearer; what the rest would add has either sign, as h's
// rounding has, so it does not pile up in a sum.  They accumulate in fp32 like any
// product here.  (h cut off too, the parts leave up to 2^-21, always of one sign; m
// rounded too, 2^-23.  4096 x 4096 x 1024 with gelu, call to call: 183 us, 185 as here,
// 188.)  Below about 2^-109 the last part is no normal bfloat16, and an operand keeps
// fewer bits.  Six 16-cycle instructions do 32 k of a block, where the fp32
// instruction takes eight of 32 cycles: the kernel took 167 us with all parts cut off
// (205 TFLOP/s) and 270 us with the fp32 instruction.
constexpr int kF32K = 32;
constexpr int kPartRow = 208;   // LDS bytes of a row: 3 parts x 32 k, and a pad that spreads 16 rows over the banks

struct Parts {
  u32x2 p[3];   // four values' h, m, l
};
__device__ __forceinline__ Parts split_parts(const u32x4& v) {
  auto high = [](float a, float b) {   // both upper halves
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
  };
  auto rest = [](float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); };
  Parts o;
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const uint32_t h = pack_bf16x2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
    const float a = __uint_as_float(v[e]) - __uint_as_float(h << 16);
    const float b = __uint_as_float(v[e + 1]) - __uint_as_float(h & 0xffff0000u);
    o.p[0][e / 2] = h;
    o.p[1][e / 2] = high(a, b);
    o.p[2][e / 2] = high(rest(a), rest(b));
  }
  return o;
}
// Four consecutive k (k4 their index / 4) of a row to LDS.
__device__ __forceinline__ void store_parts(lds_t* row, int k4, const u32x4& v) {
  typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
  const Parts o = split_parts(v);
#pragma unroll
  for (int k = 0; k < 3; ++k) *(lds_u32x2*)(row + 64 * k + 8 * k4) = o.p[k];
}

template <int S, bool PERM, bool GLU> struct RowCopy<float, S, PERM, GLU> {
  static constexpr int kBytes = 32 * S * kPartRow;
  u32x4 r[2][S];
  uint32_t off[S];
  const float* base[2];
  const float* lead;   // the passes' that pass_is_up leaves: S = 2's waves read one weight each
  int64_t ld;
  int kc4, left;       // rows of the operand from m0 on
  __device__ __forceinline__ void init(const float* p0, const float* p1, int64_t ld_, int rows, int m0, int tid) {
    ld = ld_;
    left = rows - m0;
    kc4 = (tid & 7) * 4;
    base[0] = p0 + (int64_t)m0 * ld;
    base[1] = GLU ? p1 + (int64_t)m0 * ld : base[0];
    lead = S == 2 && __builtin_amdgcn_readfirstlane(tid >> 7) ? base[1] : base[0];
#pragma unroll
    for (int q = 0; q < S; ++q) {
      const int t = (tid >> 3) + 32 * q, row = PERM ? weight_row<S, GLU>(t) : t;
      off[q] = m0 + row < rows ? (uint32_t)(((int64_t)row * ld + kc4) * 4) : kOOB;
    }
  }
  __device__ __forceinline__ void load(int h, int k0, int kext) {
    const __amdgpu_buffer_rsrc_t r0 = make_rsrc(lead + k0), r1 = make_rsrc(base[1] + k0);
    const bool in = k0 + kc4 < kext;
#pragma unroll
    for (int q = 0; q < S; ++q) r[h][q] = buf_load16(GLU && pass_is_up<S>(q) ? r1 : r0, in ? off[q] : kOOB);
  }
  // Row 16 i + lane % 16 of the half's 16 S rows, k = k0 + lane / 16.
  __device__ __forceinline__ float value(int i, int half, int k0, int kext, int lane) const {
    const int t = (half * S + i) * 16 + (lane & 15), g = lane >> 4, row = PERM ? weight_row<S, GLU>(t) : t;
    const bool in = row < left && k0 + g < kext;
    return buf_load4(make_rsrc(base[GLU && i >= S / 2] + k0), in ? (uint32_t)((row * ld + g) * 4) : kOOB);
  }
  __device__ __forceinline__ void store(int h, lds_t* buf, int tid) const {
#pragma unroll
    for (int q = 0; q < S; ++q) store_parts(buf + ((tid >> 3) + 32 * q) * kPartRow, tid & 7, r[h][q]);
  }
};

// M-contiguous operand: 4 x 4 blocks transposed in registers, thread (kc, mc)
// = (tid % 8, tid / 8); S = 2 needs half the threads.
template <int S> struct ColCopy<float, S> {
  static constexpr int kBytes = 32 * S * kPartRow;
  u32x4 r[2][4];
  uint32_t off[4];
  SegRows s;
  int m0, left;   // columns of the operand from m0 on
  __device__ __forceinline__ void init(const SegRows& rows, int cols, int m0_, int tid) {
    s = rows;
    m0 = m0_;
    left = cols - m0;
    const int k = (tid & 7) * 4, m = (tid >> 3) * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      off[e] = m < 32 * S && m0 + m < cols ? (uint32_t)(((int64_t)(k + e) * s.ld + m) * 4) : kOOB;
  }
  __device__ __forceinline__ void load(int h, int k0, int) {
    const __amdgpu_buffer_rsrc_t rs = s.rsrc<4>(k0, m0);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[h][e] = buf_load16(rs, off[e]);
  }
  __device__ __forceinline__ void store(int h, lds_t* buf, int tid) const {
    const int m = (tid >> 3) * 4;
    if (m >= 32 * S) return;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      store_parts(buf + (m + i) * kPartRow, tid & 7, u32x4{r[h][0][i], r[h][1][i], r[h][2][i], r[h][3][i]});
  }
  // As RowCopy's.  k0 is a multiple of 4, so its four k lie in one weight.
  __device__ __forceinline__ float value(int i, int half, int k0, int, int lane) const {
    const int t = (half * S + i) * 16 + (lane & 15);
    return buf_load4(s.rsrc<4>(k0, m0), t < left ? (uint32_t)(((lane >> 4) * s.ld + t) * 4) : kOOB);
  }
};

// The same sums with the fp32 matrix instruction, each wave on its own from
// global memory: what a wave with a NaN among its sums takes instead of them.
// The parts of an infinity hold a NaN (infinity less infinity), while the
// formula may give an infinity.  Its loads are a dword a lane and wait for each
// other: with nothing but NaN, N=4096, H=4096, F=4096 takes 4.0 ms forward (0.71
// with finite operands) and 4.6 ms backward (1.3).
template <int S, class CA, class CB>
__device__ __forceinline__ void gemm_wave_f32(f32x4 (&acc)[S][S], const CA& ca, int ka, const CB& cb, int kb, int K, int lane,
                                              int wave) {
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k = 0; k < K; k += 4) {
    float a[S], b[S];
#pragma unroll
    for (int i = 0; i < S; ++i) a[i] = ca.value(i, wave >> 1, k, ka, lane);
#pragma unroll
    for (int j = 0; j < S; ++j) b[j] = cb.value(j, wave & 1, k, kb, lane);
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < S; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[j], acc[i][j], 0, 0, 0);
  }
}

// One LDS buffer an operand: the next two stages' values are on their way into
// registers while this one is computed, and the CU's other workgroups run under
// the two barriers and the splitting.
template <int S, class CA, class CB>
__device__ __forceinline__ void gemm_small_f32(f32x4 (&acc)[S][S], CA& ca, int ka, CB& cb, int kb, int K,
                                               const SmallLds& L, int tid) {
  static_assert(CA::kBytes == SmallLdsSize<float, S>::kA && CB::kBytes == CA::kBytes, "the kernel's buffers");
  lds_t *const lds_a = L.p[0], *const lds_b = L.p[2];
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int frag = (lane & 15) * kPartRow + (lane >> 4) * 16;
  const lds_t* A = lds_a + (wave >> 1) * 16 * S * kPartRow + frag;
  const lds_t* B = lds_b + (wave & 1) * 16 * S * kPartRow + frag;
  const int KT = (K + kF32K - 1) / kF32K;
  auto load = [&](int h, int kt) {   // stages past K read zeros
    ca.load(h, kt * kF32K, ka);
    cb.load(h, kt * kF32K, kb);
  };
  auto stage = [&](int h, int kt) {
    ca.store(h, lds_a, tid);
    cb.store(h, lds_b, tid);
    __syncthreads();
    load(h, kt + 2);
    u32x4 b[3][S];
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
      for (int j = 0; j < S; ++j) b[k][j] = lds_load16(B + 16 * j * kPartRow + 64 * k);
#pragma unroll
    for (int k = 2; k >= 0; --k) {   // the small products first
      u32x4 a[S];
#pragma unroll
      for (int i = 0; i < S; ++i) a[i] = lds_load16(A + 16 * i * kPartRow + 64 * k);
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int l = 2 - k; l >= 0; --l)
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int j = 0; j < S; ++j) mma_frag<uint16_t>(acc[i][j], a[i], b[l][j]);
      __builtin_amdgcn_s_setprio(0);
    }
    __syncthreads();
  };
  load(0, 0);
  load(1, 1);
  for (int kt = 0; kt < KT; kt += 2) {
    stage(0, kt);
    if (kt + 1 < KT) stage(1, kt + 1);
  }
  bool nan = false;
#pragma unroll
  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int j = 0; j < S; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) nan |= acc[i][j][r] != acc[i][j][r];
  if (__ballot(nan)) gemm_wave_f32<S>(acc, ca, ka, cb, kb, K, lane, wave);
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
template <int S> __device__ __forceinline__ f32x4 block_sums(const f32x4& blk) {
  if constexpr (S == 8) return acc_read4(blk);
  else return blk;
}

}  // namespace flce
