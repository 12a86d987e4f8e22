// Kernels of the linear layer, y = act(x W^T + b) + residual, and of the gated
// product, h = act(x Wg^T + bg) * (x Wu^T + bu), with their gradients, for one
// element type T (each type is its own translation unit).
//
// Many tokens: the products run on the 256 x 256 MFMA tile routine of
// flce_device.hpp, with the activation, product and residual in the epilogue,
// while the accumulators are still in registers.  MFMA bounds them.
// Few tokens: every weight is read once for at most 64 rows of x, so HBM
// bounds the call and a kernel that streams weights runs instead.
#pragma once

#include <type_traits>

#include "layer_device.hpp"

namespace flce {

// ---------------------------------------------------------------------------
// Forward, tiles
// ---------------------------------------------------------------------------

// Workgroup w computes tiles w, w + grid, ... of the tokens x features plane
// (times the K parts).  Tokens are the MFMA rows and features its columns, in
// permuted order (tile_col_perm, glu_row): a lane holds 8 consecutive
// features of a token (gated: 4 of g and the same 4 of u), so a token's 128
// features of a wave are written as 16 adjacent 16-byte pieces (gated: 64
// features, 8-byte pieces).  16-bit: the next tile's first copies run under
// the epilogue.
//
// fp32: one tile a workgroup (a loop costs its register-staged copies 100
// spilled registers).
//
// SPLIT: the sums go to a.part in fp32 and layer_join_fwd_kernel does the rest.
template <class T, int ACT, bool GLU, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) layer_fwd_kernel(LayerFwd a) {
  FLCE_LDS(L, T);
  constexpr int FT = GLU ? kTile / 2 : kTile;   // features of a tile
  constexpr int C = GLU ? 4 : 8;                // consecutive features of a lane
  typedef typename std::conditional<GLU, DmaGlu, Dma<true>>::type DB;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int g = lane >> 4, c = lane & 15;
  const int tiles = a.TM * a.TN, total = tiles * a.parts;
  int n0, f0, k0;
  auto place = [&](int t) {
    const int part = SPLIT ? t / tiles : 0;
    int tm, tn;
    tile_coords(t - part * tiles, tiles, a.TM, a.TN, tm, tn);
    n0 = tm * kTile;
    f0 = tn * FT;
    k0 = part * a.kc;
  };
  auto opa = [&]() { return Opnd<T>{(const T*)a.x + k0, a.H, a.N, min(a.kc, a.H - k0)}; };
  auto opb = [&]() { return Opnd<T>{(const T*)a.W[0] + k0, a.H, a.F, min(a.kc, a.H - k0)}; };
  TileCopy<true, true, Dma<true>, DB> tc;
  auto begin = [&]() {
    const Opnd<T> A = opa(), B = opb();
    tc.da.init(A, n0, tid);
    if constexpr (GLU) tc.db.init(B.p, (const T*)a.W[1] + k0, B.ld, a.F, f0, tid);
    else tc.db.init(B, f0, tid, 2);
    tc.begin(A, B, L, tid);
  };
  int t = blockIdx.x;
  place(t);
  if constexpr (sizeof(T) == 2) {
    begin();
    __builtin_amdgcn_s_waitcnt(waitcnt_vm_lgkm0<0>());   // the mainloop's first wait allows the epilogue's stores
  }
  const bool vec = a.F % C == 0;   // whole 16-byte (gated: 8-byte) pieces of a row, all aligned
  Acc acc;
  while (true) {
    const Opnd<T> A = opa(), B = opb();
    const int fl = GLU ? wn * 64 + 4 * c : wn * kWaveTile + 8 * c;
    const int n0w = n0 + wm * kWaveTile, f = f0 + fl, part = SPLIT ? t / tiles : 0;
    const int left = a.F - f;   // features of this lane's run inside the row
    float b0[C], b1[C];
    if constexpr (!SPLIT) {
#pragma unroll
      for (int e = 0; e < C; ++e) {
        b0[e] = (a.b[0] && e < left) ? load1<T>((const T*)a.b[0] + f + e) : 0.f;
        b1[e] = (GLU && a.b[1] && e < left) ? load1<T>((const T*)a.b[1] + f + e) : 0.f;
      }
    }
    t += gridDim.x;
    const bool more = sizeof(T) == 2 && t < total;
    if constexpr (sizeof(T) == 2) {
      // Each tile's epilogue stores at least 32 times per wave, after the next tile's first copies.
      gemm_tile_bf16_run<true, true, 32>(acc, A, B, A.kext, L, tid, tc);
      if (more) {
        place(t);
        begin();
      }
    } else {
      Stager<float, true> sa;
      sa.init(A, n0, tid);
      if constexpr (GLU) {
        StagerGlu sb;
        sb.init(B.p, (const T*)a.W[1] + k0, B.ld, a.F, f0, tid);
        gemm_tile_f32_run(acc, A, sa, B, sb, A.kext, L, tid);
      } else {
        Stager<float, true> sb;
        sb.init(B, f0, tid, true);
        gemm_tile_f32_run(acc, A, sa, B, sb, A.kext, L, tid);
      }
    }
    acc_drain();
    if constexpr (SPLIT) {
      // 8 consecutive sums (gated: 4 and 4); rows are padded to 8 columns.
      const int64_t row0 = (int64_t)part * a.N + n0w;
      const __amdgpu_buffer_rsrc_t r0 = make_rsrc(a.part + row0 * a.ldp);
      const __amdgpu_buffer_rsrc_t r1 = GLU ? make_rsrc(a.part + row0 * a.ldp + a.ldp / 2) : r0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        f32x4 z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = acc_read4(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int nl = 16 * i + 4 * g + r;
          const uint32_t off = (n0w + nl < a.N && left > 0) ? (uint32_t)(nl * a.ldp + f) * 4u : kOOB;
          const float lo[4] = {z[0][r], z[1][r], z[2][r], z[3][r]}, hi[4] = {z[4][r], z[5][r], z[6][r], z[7][r]};
          buf_store_vec<float, 4>(r0, off, lo, true, 4);
          buf_store_vec<float, 4>(r1, GLU ? off : off + 16, hi, true, 4);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      // Descriptors start at the wave's first token, so offsets stay below 128 * F * 4 bytes.
      const int64_t base = (int64_t)n0w * a.F;
      const __amdgpu_buffer_rsrc_t ry = make_rsrc((const T*)a.y + base);
      const __amdgpu_buffer_rsrc_t rr = make_rsrc((const T*)a.residual + base);
      const __amdgpu_buffer_rsrc_t rz0 = make_rsrc((const T*)a.z[0] + base);
      const __amdgpu_buffer_rsrc_t rz1 = make_rsrc((const T*)a.z[1] + base);
      const bool res = !GLU && a.residual != nullptr, keep = a.z[0] != nullptr;
      auto offset = [&](int i, int r) -> uint32_t {
        const int nl = 16 * i + 4 * g + r;
        return (n0w + nl < a.N && left > 0) ? (uint32_t)(nl * a.F + f) * (uint32_t)sizeof(T) : kOOB;
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float rs[4][C];
        if (res) {
#pragma unroll
          for (int r = 0; r < 4; ++r) buf_load_vec<T, C>(rr, offset(i, r), rs[r], vec, left);
        }
        f32x4 z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = acc_read4(acc[i][j]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const uint32_t off = offset(i, r);
          float z0[C], z1[C], v[C];
#pragma unroll
          for (int e = 0; e < C; ++e) {
            z0[e] = z[e][r] + b0[e];
            if constexpr (GLU) z1[e] = z[4 + e][r] + b1[e];
          }
          if (keep) {
            buf_store_vec<T, C>(rz0, off, z0, vec, left);
            if constexpr (GLU) buf_store_vec<T, C>(rz1, off, z1, vec, left);
          }
#pragma unroll
          for (int e = 0; e < C; ++e) {
            v[e] = act_fwd<T, ACT>(z0[e]);
            if constexpr (GLU) v[e] *= z1[e];
            if (res) v[e] += rs[r][e];
          }
          buf_store_vec<T, C>(ry, off, v, vec, left);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (!more) break;
  }
}

// The epilogue of a split forward: thread i takes 8 features of one token.
template <class T, bool GLU> __global__ void __launch_bounds__(256) layer_join_fwd_kernel(LayerFwd a) {
  const int F8 = (a.F + 7) / 8;
  const bool vec = a.F % 8 == 0;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)a.N * F8; i += (int64_t)gridDim.x * 256) {
    const int n = (int)(i / F8), f = (int)(i - (int64_t)n * F8) * 8;
    const int left = min(8, a.F - f);
    float z0[8] = {}, z1[8] = {}, v[8];
    for (int p = 0; p < a.parts; ++p) {
      const float* s = a.part + ((int64_t)p * a.N + n) * a.ldp + f;
      load_vec<float, 8>(s, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) z0[e] += v[e];
      if constexpr (GLU) {
        load_vec<float, 8>(s + a.ldp / 2, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) z1[e] += v[e];
      }
    }
    const int64_t o = (int64_t)n * a.F + f;
    float rs[8] = {};
    if (!GLU && a.residual) {
      if (vec) load_vec<T, 8>((const T*)a.residual + o, rs);
      else for (int e = 0; e < left; ++e) rs[e] = load1<T>((const T*)a.residual + o + e);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e < left) {
        if (a.b[0]) z0[e] += load1<T>((const T*)a.b[0] + f + e);
        if (GLU && a.b[1]) z1[e] += load1<T>((const T*)a.b[1] + f + e);
      }
      v[e] = act_fwd_rt<T>(a.act, z0[e]);
      v[e] = GLU ? v[e] * z1[e] : v[e] + rs[e];
    }
    if (vec) {
      if (a.z[0]) store_vec<T, 8>((T*)a.z[0] + o, z0);
      if (GLU && a.z[1]) store_vec<T, 8>((T*)a.z[1] + o, z1);
      store_vec<T, 8>((T*)a.y + o, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e >= left) continue;
        if (a.z[0]) store1<T>((T*)a.z[0] + o + e, z0[e]);
        if (GLU && a.z[1]) store1<T>((T*)a.z[1] + o + e, z1[e]);
        store1<T>((T*)a.y + o + e, v[e]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Forward, few tokens
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

constexpr int kSkinnyWaves = 8;

// Workgroup b computes features 16 b .. 16 b + 15 of at most 16 TB tokens.
// Its 8 waves split K; each loads its weight rows straight into registers (no
// two waves share a weight, so LDS would only add a hop) with two groups of
// kU loads in flight, and x's rows through the caches.  The waves' sums meet
// in LDS and are added in wave order.
template <class T, bool GLU, int TB>
__global__ void __launch_bounds__(64 * kSkinnyWaves) layer_fwd_skinny_kernel(LayerFwd a) {
  constexpr int R = GLU ? 2 : 1, ES = sizeof(T);
  constexpr int kStep = 64 / ES;   // K of one step: 16 bytes in each of the 4 lane groups
  constexpr int kU = 4;
  __shared__ f32x4 red[kSkinnyWaves][R * TB][64];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, rl = lane & 15, f0 = blockIdx.x * 16;
  // Rows past F or N repeat the last one: their sums are not stored.
  const uint32_t offw = (uint32_t)min(rl, a.F - 1 - f0) * (uint32_t)(a.H * ES) + 16u * g;
  uint32_t offx[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) offx[t] = (uint32_t)min(16 * t + rl, a.N - 1) * (uint32_t)(a.H * ES) + 16u * g;
  __amdgpu_buffer_rsrc_t rw[R];
#pragma unroll
  for (int r = 0; r < R; ++r) rw[r] = make_rsrc((const T*)a.W[r] + (int64_t)f0 * a.H);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(a.x);

  const int steps = (a.H + kStep - 1) / kStep, per = (steps + kSkinnyWaves - 1) / kSkinnyWaves;
  const int s0 = wave * per, s1 = min(steps, s0 + per);
  const int klim = min(s1 * kStep, a.H) - g * (16 / ES);   // step s of this lane is inside K when s * kStep < klim
  f32x4 acc[R][TB] = {};
  u32x4 w[2][kU][R], x[2][kU][TB];
  auto load = [&](int h, int s) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const bool in = (s + u) * kStep < klim;
      const int so = 64 * (s + u);
#pragma unroll
      for (int r = 0; r < R; ++r)
        w[h][u][r] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rw[r], in ? offw : kOOB, so, 0));
#pragma unroll
      for (int t = 0; t < TB; ++t)
        x[h][u][t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, in ? offx[t] : kOOB, so, 0));
    }
  };
  auto mma = [&](int h) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) mma_frag<T>(acc[r][t], w[h][u][r], x[h][u][t]);
  };
  load(0, s0);
  for (int s = s0; s < s1; s += 2 * kU) {
    load(1, s + kU);
    mma(0);
    load(0, s + 2 * kU);
    mma(1);
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < TB; ++t) red[wave][r * TB + t][lane] = acc[r][t];
  __syncthreads();
  // Element (token n, feature f) sits in lane 16 (f / 4) + n % 16, value f % 4, of block n / 16.
  for (int i = tid; i < 256 * TB; i += 64 * kSkinnyWaves) {
    const int f = i & 15, n = i >> 4;
    if (n >= a.N || f0 + f >= a.F) continue;
    float z[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      z[r] = 0.f;
#pragma unroll
      for (int q = 0; q < kSkinnyWaves; ++q)
        z[r] += ((const float*)&red[q][r * TB + (n >> 4)][16 * (f >> 2) + (n & 15)])[f & 3];
      if (a.b[r]) z[r] += load1<T>((const T*)a.b[r] + f0 + f);
    }
    const int64_t o = (int64_t)n * a.F + f0 + f;
    float v = act_fwd_rt<T>(a.act, z[0]);
    if constexpr (GLU) v *= z[R - 1];
    else if (a.residual) v += load1<T>((const T*)a.residual + o);
    if (a.z[0]) {
      store1<T>((T*)a.z[0] + o, z[0]);
      if constexpr (GLU) store1<T>((T*)a.z[1] + o, z[R - 1]);
    }
    store1<T>((T*)a.y + o, v);
  }
}

template <class T, bool GLU> static void launch_skinny(const LayerFwd& a, hipStream_t st) {
  const dim3 grid((a.F + 15) / 16), blk(64 * kSkinnyWaves);
  if (a.N <= 16) FLCE_LAUNCH((layer_fwd_skinny_kernel<T, GLU, 1>), grid, blk, 0, st, a);
  else if (a.N <= 32) FLCE_LAUNCH((layer_fwd_skinny_kernel<T, GLU, 2>), grid, blk, 0, st, a);
  else FLCE_LAUNCH((layer_fwd_skinny_kernel<T, GLU, 4>), grid, blk, 0, st, a);
}

template <class T, bool GLU, int ACT> static void launch_fwd_act(const LayerFwd& a, dim3 grid, hipStream_t st) {
  FLCE_LAUNCH((layer_fwd_kernel<T, ACT, GLU, false>), grid, dim3(kThreads), 0, st, a);
}

template <class T, bool GLU> static void launch_fwd(const LayerFwd& a, hipStream_t st) {
  if (a.N <= kSkinnyTokens) return launch_skinny<T, GLU>(a, st);
  const int total = a.TM * a.TN * a.parts;
  const dim3 grid(sizeof(T) == 4 || total < kPersistGrid ? total : kPersistGrid);
  if (a.parts > 1) {
    FLCE_LAUNCH((layer_fwd_kernel<T, kActNone, GLU, true>), grid, dim3(kThreads), 0, st, a);
    const int64_t blocks = ((int64_t)a.N * ((a.F + 7) / 8) + 255) / 256;
    FLCE_LAUNCH((layer_join_fwd_kernel<T, GLU>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, a);
    return;
  }
  switch (a.act) {
    case kActRelu: return launch_fwd_act<T, GLU, kActRelu>(a, grid, st);
    case kActGelu: return launch_fwd_act<T, GLU, kActGelu>(a, grid, st);
    case kActGeluTanh: return launch_fwd_act<T, GLU, kActGeluTanh>(a, grid, st);
    case kActSilu: return launch_fwd_act<T, GLU, kActSilu>(a, grid, st);
    case kActSigmoid: return launch_fwd_act<T, GLU, kActSigmoid>(a, grid, st);
    default: return launch_fwd_act<T, GLU, kActNone>(a, grid, st);
  }
}

// ---------------------------------------------------------------------------
// Backward
// ---------------------------------------------------------------------------

// dz = dy act'(z), or dg = dh u act'(g) and du = dh act(g), into a.dz, and
// their column sums over a.db_rows tokens into a.dbp.  Thread (column group,
// row) = (tid % 32, tid / 32) walks its block's tokens 8 rows apart.  The sums
// take the values before they are rounded to T.
template <class T, int ACT, bool GLU> __global__ void __launch_bounds__(256) layer_dz_kernel(LayerBwd a) {
  constexpr int R = GLU ? 2 : 1;
  const int tid = threadIdx.x, f = (blockIdx.x * 32 + (tid & 31)) * 8;
  const int n1 = min(a.N, (int)(blockIdx.y + 1) * a.db_rows);
  const bool vec = a.F % 8 == 0;
  const int left = a.F - f;
  const int width = GLU ? a.segk : (int)a.ldz;   // columns of one weight in dz
  float sum[R][8] = {};
  if (f < width) {
#pragma unroll 2
    for (int n = blockIdx.y * a.db_rows + (tid >> 5); n < n1; n += 8) {
      const int64_t o = (int64_t)n * a.F + f;
      float dy[8] = {}, z0[8] = {}, z1[8] = {}, d[R][8];
      if (vec && left > 0) {
        load_vec<T, 8>((const T*)a.dy + o, dy);
        if (ACT != kActNone || GLU) load_vec<T, 8>((const T*)a.z[0] + o, z0);
        if (GLU) load_vec<T, 8>((const T*)a.z[1] + o, z1);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (e >= left) continue;
          dy[e] = load1<T>((const T*)a.dy + o + e);
          if (ACT != kActNone || GLU) z0[e] = load1<T>((const T*)a.z[0] + o + e);
          if (GLU) z1[e] = load1<T>((const T*)a.z[1] + o + e);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v;
        d[0][e] = act_bwd<T, ACT>(z0[e], GLU ? dy[e] * z1[e] : dy[e], v);
        if (GLU) d[R - 1][e] = dy[e] * v;
#pragma unroll
        for (int r = 0; r < R; ++r) sum[r][e] += d[r][e];
      }
      if (!a.dz_is_dy) {
#pragma unroll
        for (int r = 0; r < R; ++r) store_vec<T, 8>((T*)a.dz + (int64_t)n * a.ldz + r * a.segk + f, d[r]);
      }
    }
  }
  if (!a.dbp) return;
  __shared__ float red[R][8][256];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 8; ++e) red[r][tid >> 5][8 * (tid & 31) + e] = sum[r][e];
  __syncthreads();
  const int col = blockIdx.x * 256 + tid;
  if (col >= a.F) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float s = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) s += red[r][q][tid];
    a.dbp[blockIdx.y * a.ldb + r * (a.ldb / R) + col] = s;
  }
}

// db[m][f] = the partial sums added in block order: 64 columns a workgroup, a
// quarter of the blocks per thread.
template <class T> __global__ void __launch_bounds__(256) layer_db_kernel(LayerBwd a) {
  __shared__ float red[4][64];
  const int cl = threadIdx.x & 63, q = threadIdx.x >> 6, f = blockIdx.x * 64 + cl, m = blockIdx.y;
  const float* p = a.dbp + m * (a.ldb / a.nmat) + f;
  float s = 0.f;
  if (f < a.F) {
#pragma unroll 4
    for (int b = q; b < a.db_blocks; b += 4) s += p[b * a.ldb];
  }
  red[q][cl] = s;
  __syncthreads();
  if (q == 0 && f < a.F && a.db[m]) store1<T>((T*)a.db[m] + f, (red[0][cl] + red[1][cl]) + (red[2][cl] + red[3][cl]));
}

// dx[n][h] = sum over the rows f of W (gated: of Wg, then of Wu) of
// dz[n][f] W[f][h]: C[h][n], so a lane holds four consecutive h of a token.
// Workgroup b computes tile b % G over part b / G of K.
template <class T, bool SPLIT> __global__ void __launch_bounds__(kThreads, 1) layer_dx_kernel(LayerBwd a, int TH, int TM) {
  FLCE_LDS(L, T);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int G = TH * TM, part = SPLIT ? blockIdx.x / G : 0;
  int tm, tn;
  tile_coords(blockIdx.x - part * G, G, TH, TM, tm, tn);
  const int h0 = tm * kTile, n0 = tn * kTile, k0 = part * a.dx_kc;
  const int K = max(1, min(a.dx_kc, (int)a.ldz - k0));
  const SegRows rows{{a.W[0], a.W[1]}, a.H, a.F, a.segk, k0};
  const Opnd<T> A{(const T*)a.W[0], a.H, a.H, K};   // K only: rows past F read zeros
  const Opnd<T> B{(const T*)a.dz + k0, a.ldz, a.N, (int)a.ldz - k0};
  Acc acc;
  if constexpr (sizeof(T) == 2) {
    TileCopy<false, true, DmaSeg, Dma<true>> tc;
    tc.da.d.init(A, h0, tid);
    tc.da.s = rows;
    tc.da.m0 = h0;
    tc.db.init(B, n0, tid);
    tc.begin(A, B, L, tid);
    gemm_tile_bf16_run<false, true>(acc, A, B, K, L, tid, tc);
  } else {
    StagerSeg sa;
    sa.st.init(A, h0, tid);
    sa.s = rows;
    sa.m0 = h0;
    Stager<float, true> sb;
    sb.init(B, n0, tid);
    gemm_tile_f32_run(acc, A, sa, B, sb, K, L, tid);
  }
  acc_drain();
  const int g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = n0 + wn * kWaveTile + 16 * j + (lane & 15);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x4 z = acc_read4(acc[i][j]);
      const int h = h0 + wm * kWaveTile + 16 * i + 4 * g;
      if (n < a.N && h < a.H) {
        if constexpr (SPLIT) *(f32x4*)(a.part + ((int64_t)part * a.N + n) * a.H + h) = z;
        else store4<T>((T*)a.dx + (int64_t)n * a.H + h, z[0], z[1], z[2], z[3]);
      }
    }
  }
}

// dW[f][h] = sum_n dz[n][f] x[n][h]: C[h][f].  Column tile tn belongs to
// weight m0 + tn / TF.  SPLIT: part b / G of the tokens.
template <class T, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) layer_dw_kernel(LayerBwd a, int TH, int TF, int m0, int mats) {
  FLCE_LDS(L, T);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wm = wave >> 1, wn = wave & 1;
  const int G = TH * TF * mats, part = SPLIT ? blockIdx.x / G : 0;
  int tm, tn;
  tile_coords(blockIdx.x - part * G, G, TH, TF * mats, tm, tn);
  const int m = m0 + tn / TF;
  const int h0 = tm * kTile, f0 = (tn - (m - m0) * TF) * kTile, k0 = part * a.dw_kc;
  const int K = min(a.dw_kc, a.N - k0);
  const int width = a.nmat == 2 ? a.segk : (int)a.ldz;
  const Opnd<T> A{(const T*)a.x + (int64_t)k0 * a.H, a.H, a.H, max(K, 0)};
  const Opnd<T> B{(const T*)a.dz + (int64_t)k0 * a.ldz + (m ? a.segk : 0), a.ldz, width, max(K, 0)};
  Acc acc;
  gemm_tile<T, false, false>(acc, A, h0, B, f0, max(K, 1), L, tid);   // K >= 1: no token sums zeros
  acc_drain();
  const int g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int f = f0 + wn * kWaveTile + 16 * j + (lane & 15);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const f32x4 z = acc_read4(acc[i][j]);
      const int h = h0 + wm * kWaveTile + 16 * i + 4 * g;
      if (f < a.F && h < a.H) {
        if constexpr (SPLIT) *(f32x4*)(a.part + (((int64_t)part * mats + (m - m0)) * a.F + f) * a.H + h) = z;
        else store4<T>((T*)a.dW[m] + (int64_t)f * a.H + h, z[0], z[1], z[2], z[3]);
      }
    }
  }
}

// A split product's parts added in part order: n values to d0, and the n
// after them in each part to d1 if there is one.  Four values a thread.
template <class T>
__global__ void __launch_bounds__(256) layer_join_kernel(const float* part, int parts, int64_t n, T* d0, T* d1) {
  const int64_t all = d1 ? 2 * n : n;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < all; i += (int64_t)gridDim.x * 1024) {
    f32x4 v = *(const f32x4*)(part + i);
    for (int p = 1; p < parts; ++p) v += *(const f32x4*)(part + p * all + i);
    store4<T>(i < n ? d0 + i : d1 + (i - n), v[0], v[1], v[2], v[3]);
  }
}

template <class T> static void launch_join(const float* part, int parts, int64_t n, void* d0, void* d1, hipStream_t st) {
  const int64_t blocks = ((d1 ? 2 * n : n) / 4 + 255) / 256;
  FLCE_LAUNCH((layer_join_kernel<T>), dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, part, parts, n,
              (T*)d0, (T*)d1);
}

template <class T, bool GLU, int ACT> static void launch_dz_act(const LayerBwd& a, hipStream_t st) {
  const int width = GLU ? a.segk : (int)a.ldz;
  FLCE_LAUNCH((layer_dz_kernel<T, ACT, GLU>), dim3((width + 255) / 256, a.db_blocks), dim3(256), 0, st, a);
}

template <class T, bool GLU> static void launch_dz(const LayerBwd& a, hipStream_t st) {
  switch (a.act) {
    case kActRelu: return launch_dz_act<T, GLU, kActRelu>(a, st);
    case kActGelu: return launch_dz_act<T, GLU, kActGelu>(a, st);
    case kActGeluTanh: return launch_dz_act<T, GLU, kActGeluTanh>(a, st);
    case kActSilu: return launch_dz_act<T, GLU, kActSilu>(a, st);
    case kActSigmoid: return launch_dz_act<T, GLU, kActSigmoid>(a, st);
    default: return launch_dz_act<T, GLU, kActNone>(a, st);
  }
}

template <class T> static void launch_bwd(const LayerBwd& a, hipStream_t st) {
  const int TH = (a.H + kTile - 1) / kTile, TM = (a.N + kTile - 1) / kTile, TF = (a.F + kTile - 1) / kTile;
  const dim3 blk(kThreads);
  const bool want_db = a.db[0] || a.db[1];
  if (a.N > 0 && (!a.dz_is_dy || want_db)) {
    if (a.nmat == 2) launch_dz<T, true>(a, st);
    else launch_dz<T, false>(a, st);
  }
  if (want_db) FLCE_LAUNCH((layer_db_kernel<T>), dim3((a.F + 63) / 64, a.nmat), dim3(256), 0, st, a);
  if (a.dx && a.N > 0) {
    if (a.dx_parts > 1) {
      FLCE_LAUNCH((layer_dx_kernel<T, true>), dim3(TH * TM * a.dx_parts), blk, 0, st, a, TH, TM);
      launch_join<T>(a.part, a.dx_parts, (int64_t)a.N * a.H, a.dx, nullptr, st);
    } else {
      FLCE_LAUNCH((layer_dx_kernel<T, false>), dim3(TH * TM), blk, 0, st, a, TH, TM);
    }
  }
  if (a.dW[0] || a.dW[1]) {
    const int m0 = a.dW[0] ? 0 : 1, mats = (a.dW[0] && a.dW[1]) ? 2 : 1;
    const int G = TH * TF * mats;
    if (a.dw_parts > 1) {
      FLCE_LAUNCH((layer_dw_kernel<T, true>), dim3(G * a.dw_parts), blk, 0, st, a, TH, TF, m0, mats);
      launch_join<T>(a.part, a.dw_parts, (int64_t)a.F * a.H, a.dW[m0], mats == 2 ? a.dW[1] : nullptr, st);
    } else {
      FLCE_LAUNCH((layer_dw_kernel<T, false>), dim3(G), blk, 0, st, a, TH, TF, m0, mats);
    }
  }
}

template <class T> static hipError_t layer_forward(const LayerFwd& a, hipStream_t st) {
  if (a.nmat == 2) launch_fwd<T, true>(a, st);
  else launch_fwd<T, false>(a, st);
  return hipGetLastError();
}
template <class T> static hipError_t layer_backward(const LayerBwd& a, hipStream_t st) {
  launch_bwd<T>(a, st);
  return hipGetLastError();
}

}  // namespace flce
