// vla_layer.cu -- the translation unit of include/vla_layer.h: the operators
// are in the headers below, kernels and entry points together.
#include "vla_decay_host.cuh"
#include "vla_norm.cuh"
#include "vla_state.cuh"
