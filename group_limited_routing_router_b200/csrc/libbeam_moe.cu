// The library's one translation unit (the status word and the device set-up exist once): the layer's entry
// points, then the operators of their own.
#include "beam_moe.cu"
#include "ragged_api.cuh"
