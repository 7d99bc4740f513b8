// Element access shared by the log-probability and embedding kernels (internal; not part of the C
// ABI): 16-byte vectors at any element alignment, rounding to bf16, and the size of a launch.
#pragma once

#include "step_common.h"

namespace dllm {

// A 16-byte vector of a row that is aligned to its element type only: the hardware reads and writes
// unaligned vectors, so odd strides and bases take the same path as aligned ones.
template <bool BF16>
struct Row;
template <>
struct Row<true> {
    typedef u32x4 vec __attribute__((aligned(2)));
};
template <>
struct Row<false> {
    typedef u32x4 vec __attribute__((aligned(4)));
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Two floats to bf16, to nearest even: the one rounding of a result held in 32 bits until then.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const f32x2 v = {a, b};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Host: whether a launch of this many workgroups fits: a dimension of a grid holds fewer than 2^32 threads.
inline bool launchable(int64_t blocks, int64_t threads) { return blocks * threads < (int64_t)1 << 32; }

// Lane i reads lane i-1; lane 0 keeps its own.  Every lane must be active.
__device__ __forceinline__ int up_one(int v) { return wave_dpp::mov<0x138>(v, v); }

}  // namespace dllm
