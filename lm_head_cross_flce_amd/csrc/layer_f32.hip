// The feed-forward operators' kernels for f32 tensors.
#include "layer_kernels.hpp"

namespace flce {

hipError_t layer_pad_f32(const LayerPad& a, hipStream_t st) { return layer_pad<float>(a, st); }
hipError_t layer_forward_f32(const LayerFwd& a, hipStream_t st) { return layer_forward<float>(a, st); }
hipError_t layer_backward_f32(const LayerBwd& a, hipStream_t st) { return layer_backward<float>(a, st); }

}  // namespace flce
