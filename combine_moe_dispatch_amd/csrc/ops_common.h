// Device helpers shared by the operators around dispatch and combine (norm,
// routing, the experts' products, the few-token layer).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace ops {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int WAVE = 64;
constexpr int SCALE_BLOCK = 128;      // elements per scale, rows; also rows per weight scale block

__device__ inline float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ inline float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// Two fp32 values to packed bf16, round to nearest even; NaN stays NaN.
__device__ inline uint32_t bf16_pack(float lo, float hi)
{
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    const v2b v = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(uint32_t, v);
}

// The largest of 16 consecutive lanes, in each of them (rotations inside the
// vector unit, no LDS).
template <int N>
__device__ inline float rotate16(float v)
{
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x120 + N, 0xF, 0xF, true));
}
__device__ inline float max16(float v)
{
    v = fmaxf(v, rotate16<8>(v));
    v = fmaxf(v, rotate16<4>(v));
    v = fmaxf(v, rotate16<2>(v));
    return fmaxf(v, rotate16<1>(v));
}

// The largest of a wave's unsigned values, and the sum of its floats (in a
// fixed order), as uniform values: rotations inside rows of 16 lanes, then
// row 0 into row 1 and row 2 into row 3, then row 1 into row 3.
template <int CTRL, int ROWS>
__device__ inline uint32_t move_rows(uint32_t v)      // 0 in the rows that take nothing
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, ROWS == 0xF);
}
__device__ inline uint32_t wave_max(uint32_t v)
{
    v = max(v, move_rows<0x128, 0xF>(v));
    v = max(v, move_rows<0x124, 0xF>(v));
    v = max(v, move_rows<0x122, 0xF>(v));
    v = max(v, move_rows<0x121, 0xF>(v));
    v = max(v, move_rows<0x142, 0xA>(v));
    v = max(v, move_rows<0x143, 0xC>(v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, WAVE - 1);
}
// Inclusive sum over the lanes up to and with this one.
__device__ inline int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);       // row shifts by 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += (int)move_rows<0x142, 0xA>((uint32_t)v);
    v += (int)move_rows<0x143, 0xC>((uint32_t)v);
    return v;
}
__device__ inline float wave_sum(float v)
{
    v += rotate16<8>(v);
    v += rotate16<4>(v);
    v += rotate16<2>(v);
    v += rotate16<1>(v);
    v += __uint_as_float(move_rows<0x142, 0xA>(__float_as_uint(v)));
    v += __uint_as_float(move_rows<0x143, 0xC>(__float_as_uint(v)));
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), WAVE - 1));
}

// c exp(x), c a power of two.  The exponential instruction is of base 2: x
// log2(e) rounded to fp32 would leave an error of |x| 2^-24 in the result, so
// what that rounding and the constant's lose, r, goes into it as 2^r = 1 + r ln
// 2.  Off by four roundings of 2^-24, zero where exp(x) is below the normal
// numbers, +infinity above the largest; infinities as -200 and 200, NaN as -200.
__device__ inline float exp_of(float x, float c = 1.0f)
{
    constexpr double LOG2E = 1.4426950408889634074;
    constexpr float HI = (float)LOG2E, LO = (float)(LOG2E - HI);
    x = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
    const float t = x * HI;
    const float r = fmaf(x, LO, fmaf(x, HI, -t));
    return __builtin_amdgcn_exp2f(t) * fmaf(r, 0.69314718f * c, c);
}

// Four times silu(v) = v / (1 + exp(-v)), the same for every operator that
// forms it; the factor is the caller's to take out, where it costs least.  The
// reciprocal instruction gives zero for results below the normal numbers, that
// is for 1 + exp(-v) above 2^126 (v below -87.3); for a quarter of it, never.
// It is off by one place of 2^-23 at most.  gate/up of 16 experts, 16384 rows, f
// 4096, k 512, where the activation weighs most: 217 us, 207 with the plain
// exponential, 238-242 with a division by the letter.  NaN stays NaN.
__device__ inline float silu4(float v) { return v * __builtin_amdgcn_rcpf(exp_of(-v, 0.25f) + 0.25f); }

// The dispatch payload's block scale from a block's largest magnitude:
// scale = amax/448 and inv = 448/amax (correctly rounded divisions), the
// scale held at the smallest normal number, 1 for a block of zeros.
__device__ inline void block_scale(float amax, float& inv, float& scale)
{
    inv = 0.0f;
    scale = 1.0f;
    if (amax >= 0x1.cp-118f) {             // 448 * 2^-126
        inv = 448.0f / amax;
        scale = amax / 448.0f;
    } else if (amax > 0.0f) {
        inv = 0x1p126f;
        scale = 0x1p-126f;
    }
}

// Four fp32 values to four e4m3 codes (first in the low byte), round to
// nearest even.  The values are a block's, times its inverse scale: finite
// ones are at most 448 but for the roundings of the inverse and the product,
// far below 464 where the conversion would leave the format; NaN codes as NaN.
__device__ inline uint32_t e4m3_pack4(float a, float b, float c, float d)
{
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return (uint32_t)r;
}

// Eight e4m3 codes (two dwords) as fp16, exactly: the format's values
// (2^-9 .. 448, NaN) are all normal fp16 numbers.  The instruction
// takes two codes at the rate of an fp32 add.
__device__ inline v8h e4m3_to_f16(uint32_t lo, uint32_t hi)
{
    const v2h a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, false);
    const v2h b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, true);
    const v2h c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, false);
    const v2h d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, true);
    return v8h{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

}  // namespace ops
}  // namespace moe
