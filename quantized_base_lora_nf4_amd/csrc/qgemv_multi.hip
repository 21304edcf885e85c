// The few-token kernels of gemv.hip for rows of many adapters.
#define QN_GEMV_MULTI
#include "gemv.hip"
