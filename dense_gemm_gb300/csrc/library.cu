// The library's one translation unit: the GEMM entry points and the operators
// around them share their device status words and host helpers.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "gemm_f16.cu"
#include "ops.cu"
