// The library as one translation unit: the device word of the index checks
// (check.cuh) has one copy that every kernel and awq_bounds_error share.
#include "awq_api.cu"
#include "serve_api.cuh"
