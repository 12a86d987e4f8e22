// Launch interface of the norm, the microscaled tensors and the sampler.
// The launchers are declared weak: a build of the host code alone (under a
// sanitizer) links without them.
#pragma once

#include "flce_launch.hpp"

namespace flce {

#define FLCE_WEAK __attribute__((weak))

// Microscaled formats; a tensor's columns are padded to kMxPad.
enum MxFormat { kMxE4M3 = 0, kMxE2M1 = 1 };
constexpr int kMxBlock = 32, kMxPad = 128;

// ---------------------------------------------------------------------------
// Root-mean-square norm
// ---------------------------------------------------------------------------

struct NormFwd {
  const void* x; const void* residual; const void* weight;   // [N][H], [N][H] or null, [H] or null
  void* h;                 // [N][H]: x + residual, or null
  void* y;                 // [N][H], or null
  uint8_t* codes; uint8_t* scales;   // microscaled output instead of y, or null
  float* rstd;             // [N], or null
  int64_t N;
  int H, Hp;               // Hp: H rounded up to kMxPad
  int format;
  float eps;
  int blocks;
};

struct NormBwd {
  const void* h; const void* weight; const float* rstd; const void* dy; const void* dh;   // weight, dh may be null
  void* dx; void* dweight;   // either may be null
  float* part;               // [parts][H] fp32 sums for dweight
  int64_t N;
  int H;
  int parts;                 // workgroups: p takes groups of rows p, p + parts, ...
};

// Columns that a row's lanes hold in registers; longer rows are walked twice.
constexpr int kNormMost = 16384;
// Lanes of a row (8 columns a lane at a time, as few lanes as keep a row's share of
// registers small; 8 lanes: eight rows a wave; a microscaled row has 128 columns at
// least) and rows of a workgroup.
constexpr int norm_lanes(int width, bool mx) { return width <= 64 && !mx ? 8 : width <= 1024 ? 64 : width <= 8192 ? 256 : 1024; }
constexpr int norm_rows(int lanes) { return lanes < 256 ? 256 / lanes : 1; }

FLCE_WEAK hipError_t launch_rms_norm_forward(const NormFwd& a, int dtype, hipStream_t st);
FLCE_WEAK hipError_t launch_rms_norm_backward(const NormBwd& a, int dtype, hipStream_t st);

// ---------------------------------------------------------------------------
// Microscaled tensors
// ---------------------------------------------------------------------------

struct MxConvert {
  const void* x;                     // quantise: [R][C]
  void* y;                           // dequantise: [R][C]
  uint8_t* codes; uint8_t* scales;   // [R][Cp] or [R][Cp / 2], [R][Cp / 32]
  int64_t R;
  int C, Cp;
  int format;
};

FLCE_WEAK hipError_t launch_mx_quantize(const MxConvert& a, int dtype, hipStream_t st);
FLCE_WEAK hipError_t launch_mx_dequantize(const MxConvert& a, int dtype, hipStream_t st);

struct MxLinear {
  const uint8_t* x; const uint8_t* xs;   // codes and scales of [N][Kp]
  const uint8_t* W; const uint8_t* Ws;   // of [F][Kp], e2m1
  const void* b; const void* residual;   // [F], [N][F], or null
  void* y;                               // [N][F]
  int N, F, Kp;
  int format;                            // of x
  int act;
  int tile;                // S of the 32 S x 32 S output tiles; 0: the few-token kernel; 1: its wide form
  int TM, TN;
  int parts, kc;           // K split: parts of kc columns each
  float* part;             // parts > 1: [parts][N][ldp] fp32 sums
  int64_t ldp;
};

FLCE_WEAK hipError_t launch_mx_linear(const MxLinear& a, int dtype, hipStream_t st);

// The 256-row tile's scales come 16 bytes of a row at a time, for four steps of 128 columns.  The first byte of the run
// for the four steps from column `first` on, of a row of `bytes` (16 or more) scales: a row's last run ends with it.
constexpr int mx_scale_run(int first, int bytes) { return first / kMxBlock < bytes - 16 ? first / kMxBlock : bytes - 16; }
// Where in that run the four bytes of the step at column k lie.  A step past the row (the second of a pair, with an odd
// number of steps) has none: it is given the last four, so that it reads inside the run too.
constexpr int mx_scale_place(int k, int first, int bytes) {
  const int at = k / kMxBlock - mx_scale_run(first, bytes);
  return at < 12 ? at : 12;
}

// ---------------------------------------------------------------------------
// Sampling
// ---------------------------------------------------------------------------

struct Sample {
  const void* logits;      // [N][V]
  const float* u;          // [N]
  const float* temperature; const int64_t* top_k; const float* top_p; const float* min_p;   // [N] or null
  float temperature0; int64_t top_k0; float top_p0; float min_p0;   // where those are null
  int64_t* tokens;         // [N]
  int64_t N;
  int V;
  // Rows of more than kOneLaunchTokens: what a first launch finds of each row's slices and groups.
  int slices, groups;      // slices 0: one launch does it all
  uint32_t* group_top;     // [N][groups]: the largest of each kGroupTokens tokens, as value_key
  uint32_t* slice_top;     // [N][slices], of each kSliceTokens
  double* slice_sum;       // [N][slices]: sum of exp((z - largest) / T), for rows that need it
  // Rows with top-p and without top-k: each slice's histogram of exp(z / T), kHistBins bins from slice_bin on.
  int* slice_bin;          // [N][slices]
  unsigned long long* hist;   // [N][slices][kHistBins]
  int hist_shift;          // in whole numbers of 2^-hist_shift
};
constexpr int kGroupTokens = 32, kSliceTokens = 8192, kOneLaunchTokens = 8192, kHistBins = 512;

FLCE_WEAK hipError_t launch_sample(const Sample& a, int dtype, hipStream_t st);

}  // namespace flce
