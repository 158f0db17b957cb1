// The input gradient of a linear layer, BF16.
#include "ecf8_product.cuh"

template int ecf8_linear_impl::product_launch<__nv_bfloat16, 1>(bool, const CUtensorMap&, const CUtensorMap&,
                                                                const ecf8_linear_impl::ProductArgs&, dim3, size_t, bool,
                                                                cudaStream_t);
