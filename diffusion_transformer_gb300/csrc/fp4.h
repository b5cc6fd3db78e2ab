// Internal interface of the 4-bit matrices: what api.cu calls in fp4.cu and fp4_gemm.cu, on validated
// arguments (see dit_fp4_quantize and the calls after it).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace dit {

int fp4_quantize_launch(const void* x, int type, long long ldx, const dit_fp4_matrix& m, cudaStream_t stream);
int fp4_dequantize_launch(const dit_fp4_matrix& m, void* out, int type, long long ldo, cudaStream_t stream);

// out = a b^T. b_early: the kernel enqueued just before the product does not write b and itself called
// pdl_wait before pdl_trigger (as every kernel here does), so b was complete when the product's launch
// began; its loads may then run ahead of that kernel's end.
int fp4_matmul_launch(const dit_fp4_matrix& a, const dit_fp4_matrix& b, void* out, int type, long long ldo, int* err,
                      bool b_early, cudaStream_t stream);

// A block's linear a b^T through kEpiQKV, kEpiSwiGLU or kEpiGated (g.out, g.ldo, g.err and what the epilogue
// reads; b as with b_early), for the widths a block has: b->rows a multiple of 256.
int fp4_block_linear_launch(const dit_fp4_matrix& a, const dit_fp4_matrix& b, int epi, const GemmParams& g,
                            cudaStream_t stream);

}  // namespace dit
