// gemm_epilogue.cu -- the FP4 and fp32-scale GEMM kernels with a fused epilogue
// (bias, activation, residual): gemm.cu once more, compiled beside it.
#define UFP4_EPILOGUE_PART 1
#include "gemm.cu"
