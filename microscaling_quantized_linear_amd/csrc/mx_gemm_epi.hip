// mx_gemm_epi.hip -- the W8A8 prefill GEMM with an epilogue (mx_epilogue.h): the
// kernel of mx_gemm.hip, compiled a second time.
#define MX_WITH_EPILOGUE
#include "mx_gemm.hip"
