// The feed-forward operators' kernels for bf16 tensors.
#include "layer_kernels.hpp"

namespace flce {

hipError_t layer_pad_bf16(const LayerPad& a, hipStream_t st) { return layer_pad<uint16_t>(a, st); }
hipError_t layer_forward_bf16(const LayerFwd& a, hipStream_t st) { return layer_forward<uint16_t>(a, st); }
hipError_t layer_backward_bf16(const LayerBwd& a, hipStream_t st) { return layer_backward<uint16_t>(a, st); }

}  // namespace flce
