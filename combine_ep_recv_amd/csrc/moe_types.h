// moe_types.h -- element types, wavefront reductions and pointer checks shared by the gate and the
// microscaled kernels (gfx950, wave64).
#ifndef MOE_TYPES_H
#define MOE_TYPES_H

#include <hip/hip_runtime.h>

#include <stddef.h>
#include <stdint.h>

#include "moe_ep.h"

namespace moe_detail {

constexpr int kWave = 64;

// 16- and 32-bit element types: their raw bits, and conversion to and from fp32 (round to nearest, ties to even)
struct F16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(raw b) { return (float)__builtin_bit_cast(_Float16, b); }
    static __device__ __forceinline__ raw store(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
struct BF16 {
    using raw = uint16_t;
    static __device__ __forceinline__ float load(raw b) { return __uint_as_float((uint32_t)b << 16); }
    static __device__ __forceinline__ raw store(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
struct F32 {
    using raw = uint32_t;
    static __device__ __forceinline__ float load(raw b) { return __uint_as_float(b); }
    static __device__ __forceinline__ raw store(float f) { return __float_as_uint(f); }
};

// One DPP move (row shift or broadcast); lanes without a source get `old`.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double old, double v)
{
    const int lo = __builtin_amdgcn_update_dpp(__double2loint(old), __double2loint(v), CTRL, ROWS, 0xf, false);
    const int hi = __builtin_amdgcn_update_dpp(__double2hiint(old), __double2hiint(v), CTRL, ROWS, 0xf, false);
    return __hiloint2double(hi, lo);
}
__device__ __forceinline__ float lane_value(float v, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane)
{
    return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), lane),
                            __builtin_amdgcn_readlane(__double2loint(v), lane));
}
__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double max_of(double a, double b) { return fmax(a, b); }

// Reductions over a group of LANES lanes (the 64 of a wavefront, or each row of 16), the same value in every lane of
// the group. Every lane of the wavefront is active. The order of a sum is fixed. Each step is one instruction that
// moves and combines, behind the two cycles that a move needs after its operand was written (the compiler spends five
// instructions on it). Of 64 lanes: row shifts by 1, 2, 4 and 8 (lanes without a source keep their value), the last
// lane of a row to the rows above, then lane 63 to all. Of 16: rotations; a sum takes shifts, so that every lane gets
// the last one's.
#define MOE_REDUCE_64(op)                                                                             \
    "s_nop 1\n\t" op " %0, %0, %0 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_bcast:15 row_mask:0xa bank_mask:0xf\n\t"                       \
    "s_nop 1\n\t" op " %0, %0, %0 row_bcast:31 row_mask:0xc bank_mask:0xf\n\t"                       \
    "s_nop 1"
#define MOE_REDUCE_16(op)                                                                             \
    "s_nop 1\n\t" op " %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_ror:4 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_ror:2 row_mask:0xf bank_mask:0xf\n\t"                          \
    "s_nop 1\n\t" op " %0, %0, %0 row_ror:1 row_mask:0xf bank_mask:0xf"
template <int LANES = kWave>
__device__ __forceinline__ float wave_max(float v)
{
    if constexpr (LANES == 16) {
        asm(MOE_REDUCE_16("v_max_f32_dpp") : "+v"(v));
        return v;
    }
    asm(MOE_REDUCE_64("v_max_f32_dpp") : "+v"(v));
    return lane_value(v, 63);
}
template <int LANES = kWave>
__device__ __forceinline__ uint32_t wave_min(uint32_t v)
{
    if constexpr (LANES == 16) {
        asm(MOE_REDUCE_16("v_min_u32_dpp") : "+v"(v));
        return v;
    }
    asm(MOE_REDUCE_64("v_min_u32_dpp") : "+v"(v));
    return __builtin_amdgcn_readlane(v, 63);
}
template <int LANES = kWave>
__device__ __forceinline__ float wave_sum(float v)
{
    if constexpr (LANES == 16) {
        asm("s_nop 1\n\tv_add_f32_dpp %0, %0, %0 row_shr:1 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1\n\tv_add_f32_dpp %0, %0, %0 row_shr:2 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1\n\tv_add_f32_dpp %0, %0, %0 row_shr:4 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1\n\tv_add_f32_dpp %0, %0, %0 row_shr:8 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1\n\tv_mov_b32_dpp %0, %0 row_newbcast:15 row_mask:0xf bank_mask:0xf"
            : "+v"(v));
        return v;
    }
    asm(MOE_REDUCE_64("v_add_f32_dpp") : "+v"(v));
    return lane_value(v, 63);
}
#undef MOE_REDUCE_64
#undef MOE_REDUCE_16
// (row 0 + row 1) + (row 2 + row 3) of the wavefront's rows of 16 lanes, in every row
__device__ __forceinline__ float sum_of_rows(float v)
{
    const auto odd = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(odd[0]) + __uint_as_float(odd[1]);
    const auto half = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(half[0]) + __uint_as_float(half[1]);
}
__device__ __forceinline__ double wave_max(double v)
{
    v = max_of(v, dpp<0x111, 0xf>(v, v));
    v = max_of(v, dpp<0x112, 0xf>(v, v));
    v = max_of(v, dpp<0x114, 0xf>(v, v));
    v = max_of(v, dpp<0x118, 0xf>(v, v));
    v = max_of(v, dpp<0x142, 0xa>(v, v));
    v = max_of(v, dpp<0x143, 0xc>(v, v));
    return lane_value(v, 63);
}
__device__ __forceinline__ double wave_sum(double v)
{
    const double z = 0;
    v += dpp<0x111, 0xf>(z, v);
    v += dpp<0x112, 0xf>(z, v);
    v += dpp<0x114, 0xf>(z, v);
    v += dpp<0x118, 0xf>(z, v);
    v += dpp<0x142, 0xa>(z, v);
    v += dpp<0x143, 0xc>(z, v);
    return lane_value(v, 63);
}

// Orders a wavefront's own LDS writes before its reads of other lanes' words.
__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

inline bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

}  // namespace moe_detail

#endif  // MOE_TYPES_H
