// gemm_epilogue_mx.cu -- the MX (block-scaled FP8) GEMM kernels with a fused
// epilogue: gemm.cu once more, compiled beside it.
#define UFP4_EPILOGUE_PART 2
#include "gemm.cu"
