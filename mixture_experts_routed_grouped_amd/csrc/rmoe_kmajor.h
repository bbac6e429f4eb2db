// k-major operands: an LDS slot holds k rows of a row-major matrix whose row
// index the sum runs along, and ds_read_b64_tr_b16 turns it into MFMA
// operands: a group of 16 lanes reads 4 k rows of 16 columns and each lane
// receives its column's 4 values.
//
// Slot: [column groups of 64][k groups of 8] blocks of 1 KB = 8 rows x 128
// bytes, one DMA instruction each; 16-byte chunk c of row r sits at
// c ^ swz_k(r), which spreads the 4 rows x 64 bytes that 32 lanes read over
// all 64 banks.
#pragma once

#include "rmoe_device.h"

namespace rmoe {

typedef short s4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ int swz_k(int r) { return ((r >> 1) & 1) * 4 | ((r >> 2) & 1) * 2; }

// Lane offset in a k-major slot of read half h of a 32-column tile of parity
// tp: rows 4h .. 4h+3 of k group lane / 32 (sub-step s of 16 rows: + 2048 s).
__device__ __forceinline__ unsigned tr_off(int lane, int tp, int h) {
    const int i = lane & 15, n16 = (lane >> 4) & 1, lh = lane >> 5;
    const int r = 4 * h + (i >> 2), c = 4 * tp + 2 * n16 + ((i & 3) >> 1);
    return lh * 1024 + r * 128 + ((c ^ swz_k(r)) << 4) + (i & 1) * 8;
}
__device__ __forceinline__ h4 tr_read(const unsigned char *p) {
    return __builtin_bit_cast(
        h4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4 *)p));
}

}  // namespace rmoe
