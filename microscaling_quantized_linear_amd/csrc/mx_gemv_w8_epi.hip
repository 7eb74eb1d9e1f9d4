// mx_gemv_w8_epi.hip -- the W8A8 decode GEMVs with an epilogue (mx_epilogue.h): the
// kernels of mx_gemv_w8.hip, compiled a second time.
#define MX_WITH_EPILOGUE
#include "mx_gemv_w8.hip"
