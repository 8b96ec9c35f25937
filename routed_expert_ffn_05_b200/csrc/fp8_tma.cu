// Tensor maps of the FP8 operators' operand tiles (see fp8.h).
#include "fp8.h"
#include "tma.h"

namespace moe {

bool make_rows_map_u8(CUtensorMap *map, const void *base, uint64_t rows, uint64_t cols, uint64_t ld,
                      uint32_t box_rows) {
    if (ld % 16 || ld < cols || !cols || !rows || reinterpret_cast<uintptr_t>(base) % 16) return false;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {ld};
    const cuuint32_t box[2] = {128, box_rows};
    return encode_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace moe
