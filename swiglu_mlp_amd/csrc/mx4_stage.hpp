// mx4_stage.hpp -- where in an operand's blocked codes a stage of mx4_gemm_kernel
// reads.  Plain C++, so that every read of every tile is checked on the host
// (tests/test_host_headers.py).
#pragma once
#include <cstdint>

namespace ck {
namespace mx4 {

// Byte, from the tile's first row block on, of 1 KB block `block` of the stage
// that begins with slice `slice0`: row block block / 2 of the tile, slice block % 2.
// kb: slices of a row block; left: row blocks from the tile's first to the operand's
// last.  A tile may reach past these (operands are padded to 32 rows, tiles are up
// to 256): there the last row block is read again, for products that are not stored.
// Nothing is left to the buffer's range check, which sets the scalar offset off
// against the range before it compares.
constexpr uint32_t stage_offset(int block, int kb, int slice0, int left)
{
    const int rb = block / 2 < left ? block / 2 : left - 1;
    return (uint32_t)(rb * kb + block % 2 + slice0) * 1024u;
}

}  // namespace mx4
}  // namespace ck
