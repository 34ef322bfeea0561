// The GEMM entry points and the operators around them: one translation unit, since
// they share their device status words and host helpers. The kernels that work along
// rows without either are in ops_rows.cu.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gemm_f16.cu"
#include "ops.cu"
#include "ops_block.cu"
