// int8_tile.hpp -- the INT8 product in LDS tiles, as its callers see it.
#pragma once
#include "int8_core.hpp"

namespace fp8dp {

// For operands that rows16() accepts; tiles of 256 x 256 (wide) or 128 x 128 outputs.
int tile_i8(const char* what, fp8dp_dtype yt, const I8Args& g, bool wide, hipStream_t stream);

}  // namespace fp8dp
