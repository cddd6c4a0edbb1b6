// What the two tensor-core kernels of ffn.cuh's products share: operand maps, instruction
// descriptors and the MMAs themselves.
#pragma once

#include "ffn.cuh"
#include "sm100.cuh"

namespace qg {

// int8: s32 accumulator (2), signed operands (1). 16-bit: fp32 accumulator (1), fp16 (0) or bf16
// (1) operands. Bits 15 and 16: MN-major A and B.
template <bool I8, typename T, bool AMN, bool BMN>
__device__ __forceinline__ uint32_t ffn_instr_desc(int m, int n)
{
    constexpr uint32_t in = I8 ? 1u : (std::is_same<T, __nv_bfloat16>::value ? 1u : 0u);
    return (I8 ? 2u : 1u) << 4 | in << 7 | in << 10 | (AMN ? 1u : 0u) << 15 |
           (BMN ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

#define QG_FFN_MMA(group, kind)                                                                  \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, p;\n\t}" ::"r"( \
                     dtm),                                                                        \
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                       \
                 : "memory")

// D[dtm] (+)= A . B^T over 32 bytes of a K-major slab or 16 rows of an MN-major one
template <bool I8>
__device__ __forceinline__ void ffn_mma(uint32_t dtm, uint64_t a, uint64_t b, uint32_t idesc,
                                        uint32_t accumulate)
{
    if constexpr (I8) QG_FFN_MMA("1", "i8");
    else QG_FFN_MMA("1", "f16");
}

// the same for a CTA pair
template <bool I8>
__device__ __forceinline__ void ffn_mma_pair(uint32_t dtm, uint64_t a, uint64_t b, uint32_t idesc,
                                             uint32_t accumulate)
{
    if constexpr (I8) QG_FFN_MMA("2", "i8");
    else QG_FFN_MMA("2", "f16");
}
#undef QG_FFN_MMA

// A 16-bit or int8 matrix [rows, cols] with `pitch` bytes a row, read in boxes of 128 bytes by
// box_rows rows.
struct Matrix {
    const void *p;
    uint64_t rows, cols, pitch;
};

template <bool I8, typename T> bool map_of(CUtensorMap *m, const Matrix &x, int box_rows)
{
    const bool bf16 = std::is_same<T, __nv_bfloat16>::value;
    const CUtensorMapDataType dt =
        I8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
           : (bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16);
    return make_map(m, dt, x.p, x.cols, x.rows, x.pitch, I8 ? 128 : 64, box_rows,
                    CU_TENSOR_MAP_SWIZZLE_128B);
}

} // namespace qg
