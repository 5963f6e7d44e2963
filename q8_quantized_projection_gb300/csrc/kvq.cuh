// kvq.cuh -- the formats of quantised K/V caches, shared by the kernels that write, read
// and attend to them.
//
// A head's values are cut in blocks of 32.  Codes lie head-major, [rows][kv_heads][n_pos]
// [head_dim] (Q8_KVQ_I8: a signed byte a value; Q8_KVQ_U4: four bits, the even value's low),
// so that a head's entries are one run of memory however many heads there are (entry-major
// rows would leave a head's block words in half a 32-byte sector).  Beside them lies a 4-byte
// word a block, [rows][kv_heads][n_pos][head_dim / 32]: binary32 d of a value d * code, or
// binary16 s (low half) and m of a value m + s * code.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "q8proj.h"

namespace q8 {

// Bytes of a head's codes in one entry.
__host__ __device__ constexpr int64_t kvq_row(int kind, int64_t dim) { return kind == Q8_KVQ_U4 ? dim / 2 : dim; }

// A Q8_KVQ_U4 block's s and m.
__device__ __forceinline__ float2 kvq_scale_min(uint32_t word) {
    return __half22float2(*reinterpret_cast<const __half2*>(&word));
}

}  // namespace q8
