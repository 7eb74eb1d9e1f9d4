// mx_gemv_epi.hip -- the A16 and long-K dense GEMVs with an epilogue (mx_epilogue.h):
// the kernel of mx_gemv.hip, compiled for the launch shapes of gemv_shape.
#define MX_WITH_EPILOGUE
#include "mx_gemv.hip"
