// The forward tile kernels of qgemm.hip for rows of many adapters.
#define QN_QGEMM_MULTI
#include "qgemm.hip"
