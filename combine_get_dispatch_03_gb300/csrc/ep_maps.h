// ep_maps.h -- tensor maps of operands that kernels load with bulk tensor copies (host side).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "../../include/ep.h"

namespace ep {

enum class Element { kBf16, kFp8, kFp32 };

struct Operand {
    const void* base;
    Element element;
    int dims;
    uint64_t size[4];
    uint64_t stride[3];  // bytes
    uint32_t box[4];
};

// 128-byte swizzle; what lies outside reads as 0.  The inner extent of the box is 128 bytes.
ep_status encode(CUtensorMap* map, const Operand& o);

}  // namespace ep
