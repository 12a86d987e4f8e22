// Device pieces of the feed-forward operators (the linear layer and the gated
// product): activations with their derivatives, and the operand copies for
// the tile routine of flce_device.hpp that take rows from two weights.
#pragma once

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

// C consecutive elements (C = 4 or 8) of a 16-byte (C = 4, 16-bit: 8-byte)
// aligned address.
template <class T, int C> __device__ __forceinline__ void load_vec(const T* p, float (&v)[C]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < C; e += 4) {
      const f32x4 t = *(const f32x4*)((const float*)p + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[e + k] = t[k];
    }
  } else {
    uint32_t w[C / 2];
    if constexpr (C == 8) {
      const u32x4 t = *(const u32x4*)p;
#pragma unroll
      for (int k = 0; k < 4; ++k) w[k] = t[k];
    } else {
      const u32x2 t = *(const u32x2*)p;
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
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int e = 0; e < C; e += 4) *(f32x4*)((float*)p + e) = f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]};
  } else if constexpr (C == 8) {
    *(u32x4*)p = u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])};
  } else {
    *(u32x2*)p = u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])};
  }
}

// The same through a buffer descriptor: byte offset off, kOOB reads zeros and
// stores nothing.  vec: the C elements are aligned as above and all in the
// row or all past it; else element e moves alone, `left` of them in the row.
template <class T, int C>
__device__ __forceinline__ void buf_store_vec(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&v)[C], bool vec,
                                              int left) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < C; e += 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{v[e], v[e + 1], v[e + 2], v[e + 3]}), r,
                                               off + 4 * e, 0, 0);
    } else if constexpr (C == 8) {
      __builtin_amdgcn_raw_buffer_store_b128(
          u32x4{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])}, r, off, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3])}, r, off, 0, 0);
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e) {
      const uint32_t o = e < left ? off + (uint32_t)(sizeof(T) * e) : kOOB;
      if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), r, o, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(pack2<T>(v[e], 0.f) & 0xffffu), r, o, 0, 0);
    }
  }
}
template <class T, int C>
__device__ __forceinline__ void buf_load_vec(__amdgpu_buffer_rsrc_t r, uint32_t off, float (&v)[C], bool vec, int left) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < C; e += 4) {
        const f32x4 t = __builtin_bit_cast(f32x4, buf_load16(r, off + 4 * e));
#pragma unroll
        for (int k = 0; k < 4; ++k) v[e + k] = t[k];
      }
    } else if constexpr (C == 8) {
      const u32x4 t = buf_load16(r, off);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = h16_to_f32<T>(t[k]);
        v[2 * k + 1] = h16_to_f32<T>(t[k] >> 16);
      }
    } else {
      const u32x2 t = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        v[2 * k] = h16_to_f32<T>(t[k]);
        v[2 * k + 1] = h16_to_f32<T>(t[k] >> 16);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < C; ++e) {
      const uint32_t o = e < left ? off + (uint32_t)(sizeof(T) * e) : kOOB;
      if constexpr (sizeof(T) == 4) v[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0));
      else v[e] = h16_to_f32<T>(__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0));
    }
  }
}

// ---------------------------------------------------------------------------
// Operands over two weights
// ---------------------------------------------------------------------------

// The gated product's weight tile: 128 rows of Wg and the same 128 of Wu as
// one 256-row K-contiguous operand.  In each half of 128 tile rows, row
// 16 j + c (output column c of block j) holds row 64 half + 4 c + j % 4 of Wg
// (j < 4) or of Wu (j >= 4): a lane's eight blocks of one output row are four
// consecutive columns of g and the same four of u, so the product act(g) u
// needs no other lane.
__device__ __forceinline__ constexpr int glu_row(int t) {
  return ((t & 0x80) >> 1) | ((t & 0x0F) << 2) | ((t & 0x30) >> 4);
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
      const int row = glu_row(8 * (4 * q + wave) + (lane >> 3));
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

// fp32 form: tile row t = tid / 8 + 32 q, again bit 1 of q names the weight.
struct StagerGlu {
  u32x4 r[8];
  uint32_t off[8];
  const float* base[2];
  int kc_elem;
  __device__ __forceinline__ void init(const float* Wg, const float* Wu, int64_t ld, int F, int f0, int tid) {
    const int kc = tid & 7, rr = tid >> 3;
    kc_elem = kc * 4;
    base[0] = Wg + (int64_t)f0 * ld;
    base[1] = Wu + (int64_t)f0 * ld;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = glu_row(rr + 32 * q);
      off[q] = (f0 + row < F) ? (uint32_t)(((int64_t)row * ld + kc_elem) * 4) : kOOB;
    }
  }
  __device__ __forceinline__ void load(const Opnd<float>& o, int k0) {
    const __amdgpu_buffer_rsrc_t rg = make_rsrc(base[0] + k0), ru = make_rsrc(base[1] + k0);
    const bool kok = k0 + kc_elem < o.kext;
#pragma unroll
    for (int q = 0; q < 8; ++q) r[q] = buf_load16((q & 2) ? ru : rg, kok ? off[q] : kOOB);
  }
  __device__ __forceinline__ void store(lds_t* buf, int tid) const {
    const int kc = tid & 7, rr = tid >> 3;
#pragma unroll
    for (int q = 0; q < 8; ++q) lds_store16(buf + (rr + 32 * q) * kRowBytes + kc * 16, r[q]);
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

struct StagerSeg {
  Stager<float, false> st;
  SegRows s;
  int m0;
  __device__ __forceinline__ void load(const Opnd<float>& o, int k0) {
    const __amdgpu_buffer_rsrc_t rs = s.rsrc<4>(k0, m0);
    const int kleft = o.kext - k0 - st.krow;
#pragma unroll
    for (int i = 0; i < 8; ++i) st.r[i] = buf_load16(rs, (i & 3) < kleft ? st.off[i] : kOOB);
  }
  __device__ __forceinline__ void store(lds_t* buf, int tid) const { st.store(buf, tid); }
};

}  // namespace flce
