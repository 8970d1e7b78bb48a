// Shared declarations of the 4-bit paged cache: geometry, and how its codes
// become matrix-core operands.  Not part of the public ABI.
#pragma once

#include "host.h"
#include "q4_device.h"

namespace bconv {

struct Kv4Geom {
    int num_blocks, block_shift, kv_heads, dim;
    int dim_padded, groups, row_bytes;
    int record_bytes, v_codes, k_scales, v_scales;  // a record stays below 2^31 bytes (1024 tokens x 384 bytes)
};

// Checks a descriptor and resolves its geometry.
bconv_status_t kv4_geometry(const bconv_kv4_desc_t *d, Kv4Geom *g);

inline int dtype_size(int32_t dtype)
{
    return dtype == BCONV_F32 ? 4 : dtype == BCONV_F16 || dtype == BCONV_BF16 ? 2 : 0;
}

}  // namespace bconv
