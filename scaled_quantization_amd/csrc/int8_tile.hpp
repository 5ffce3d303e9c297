// int8_tile.hpp -- the INT8 product in LDS tiles, as its callers see it.
#pragma once
#include "int8_core.hpp"

namespace fp8dp {

// For operands that rows16() accepts.
int tile_i8(const char* what, fp8dp_dtype yt, const I8Args& g, hipStream_t stream);

}  // namespace fp8dp
