// zs_mx.hip -- microscaled 4-bit parameters (OCP MXFP4) for gfx950: the
// quantisation of fp32/fp16/bf16 rows, their values back in a 16- or 32-bit
// format (one matrix, or the shards of all ranks into a full buffer), and
// the products that read the 4-bit weight in place.
//
// A row is cut into blocks of 32 consecutive values with one scale byte b
// each, which stands for 2^(b - 127); a value is a 4-bit e2m1 code (sign,
// two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) times
// that scale.  b = 255 makes the whole block NaN.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "zero_shard.h"
#include "zs_internal.h"
#include "zs_mx_rules.h"
#include "zs_ops.h"

namespace {

using namespace zs::mx;

using zs::f32x4;
using zs::u32x4;

// ---------------------------------------------------------------------------
// Element access.  Rows may start at any element (views, odd pitches):
// vectors are loaded and stored at element alignment, which global memory
// instructions of gfx950 allow.
// ---------------------------------------------------------------------------
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct F16 {
    typedef _Float16 T;
    typedef f16x8 V8;
    static constexpr int kType = ZERO_F16;
};
struct BF16 {
    typedef __bf16 T;
    typedef bf16x8 V8;
    static constexpr int kType = ZERO_BF16;
};
struct F32 {
    typedef float T;
};

// Eight consecutive 16-bit elements, those from `valid` on as zero.
template <class Fmt>
__device__ __forceinline__ typename Fmt::V8 load8(const typename Fmt::T *p, int64_t valid) {
    if (valid >= 8)
        return __builtin_bit_cast(typename Fmt::V8, (u32x4)(*(const u32x4_a2 *)p));
    typename Fmt::V8 r;
    for (int i = 0; i < 8; i++)
        r[i] = i < valid ? p[i] : (typename Fmt::T)0.0f;
    return r;
}

// Store up to four consecutive fp32 results of a row in the output's format
// (one rounding to nearest even).
template <class T>
__device__ __forceinline__ void store4(T *y, const f32x4 &v, int64_t valid) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T4 T4u __attribute__((aligned(sizeof(T))));
    if (valid >= 4) {
        *(T4u *)y = T4{(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
    } else {
        if (valid > 0)
            y[0] = (T)v[0];
        if (valid > 1)
            y[1] = (T)v[1];
        if (valid > 2)
            y[2] = (T)v[2];
    }
}

// Call f with a null pointer of the output's type.
template <class F>
__device__ __forceinline__ void by_type(int type, F f) {
    if (type == ZERO_F32)
        f((float *)nullptr);
    else if (type == ZERO_F16)
        f((_Float16 *)nullptr);
    else
        f((__bf16 *)nullptr);
}

// The scale as fp32: exact for every byte (2^-127 is a subnormal).
__device__ __forceinline__ float scale_f32(uint32_t byte) {
    const uint32_t bits = byte == 0 ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23;
    return __uint_as_float(bits);
}

// ---------------------------------------------------------------------------
// Quantisation and values: four lanes to a block, eight elements to a lane
// (fp32 to 4 bits: eight and four).  Both stream through HBM once, 4.53 bytes
// per fp32 value in and out and 2.53 per 16-bit value out.  117,187,500 fp32
// values to 4 bits and back to fp16: nontemporal fp32 loads 169 -> 156 us,
// nontemporal 16-bit stores 169 -> 147, two blocks a lane instead of four 169
// -> 166 (one 163, but small gathers and the 64-shard one slow down), all
// three 140, and 127.5 with the fp32 kernel below (6.5 TB/s of the 827 MB both
// passes move).
// ---------------------------------------------------------------------------
constexpr uint32_t kQuantThreads = 256;
constexpr uint32_t kQuantIters = 2; // blocks per four lanes
constexpr uint32_t kQuantBlocks = kQuantThreads / 4 * kQuantIters;

// Row and block-in-row of block q of a matrix of nb blocks a row.
__device__ __forceinline__ void split_block(uint64_t q, uint64_t rows, uint64_t nb,
                                            uint64_t &row, uint64_t &blk) {
    if (rows == 1) {
        row = 0;
        blk = q;
    } else if (rows * nb <= 0xFFFFFFFFull) {
        row = (uint32_t)q / (uint32_t)nb;
        blk = (uint32_t)q - (uint32_t)row * (uint32_t)nb;
    } else {
        row = q / nb;
        blk = q - row * nb;
    }
}

__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    const uint32_t a = __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, false); // lanes 1 0 3 2
    v = a > v ? a : v;
    const uint32_t b = __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, false); // lanes 2 3 0 1
    return b > v ? b : v;
}

// The block's exponent is floor(log2 amax) - 2, so that the largest value
// lands in [4, 8) and saturates at 6; the fp32 bit pattern of amax holds it
// (a subnormal amax, or 0, clamps to 2^-127).  x times the inverse scale is
// exact wherever the code is not zero, and v_cvt_scalef32_pk_fp4_f32 rounds
// it to the nearest code, ties to even, saturating.

// fp32: eight lanes to a block and four elements to a lane, so that a wave's
// load is 1 KiB in a row (four lanes to a block read every other 16 bytes
// twice over: 117,187,500 values there and back 140 us against 127.5).
__global__ __launch_bounds__(kQuantThreads) void zs_mx_quantize_f32_kernel(
    const float *__restrict__ src, uint64_t ld_src, uint64_t rows, uint64_t cols, uint64_t nb,
    uint8_t *__restrict__ codes, uint64_t ld_codes, uint8_t *__restrict__ scales,
    uint64_t ld_scales, int32_t *flag) {
    constexpr uint32_t kIters = 2 * kQuantIters;
    const uint32_t part = threadIdx.x & 7u;
    const uint64_t q0 = (uint64_t)blockIdx.x * kQuantBlocks + threadIdx.x / 8u;
    const uint64_t total = rows * nb;
    f32x4 x[kIters];
    uint64_t row[kIters], blk[kIters];
    int bad = 0;
#pragma unroll
    for (uint32_t it = 0; it < kIters; it++) {
        const uint64_t q = q0 + it * (kQuantThreads / 8u);
        x[it] = f32x4{0, 0, 0, 0};
        if (q < total) {
            split_block(q, rows, nb, row[it], blk[it]);
            const uint64_t c = blk[it] * 32u + part * 4u;
            const float *p = src + row[it] * ld_src + c;
            if (c + 4 <= cols)
                x[it] = __builtin_nontemporal_load((const f32x4_a4 *)p);
            else
                for (int i = 0; i < 4; i++)
                    x[it][i] = c + i < cols ? p[i] : 0.0f;
        }
    }
#pragma unroll
    for (uint32_t it = 0; it < kIters; it++) {
        uint32_t amax = 0;
        for (int i = 0; i < 4; i++) {
            const uint32_t b = __float_as_uint(x[it][i]) & 0x7FFFFFFFu;
            amax = b > amax ? b : amax;
        }
        amax = quad_max(amax);
        const uint32_t other = // the block's other four lanes (half-row mirror)
            __builtin_amdgcn_update_dpp(amax, amax, 0x141, 0xF, 0xF, false);
        amax = other > amax ? other : amax;
        const uint32_t e = amax >> 23;
        uint32_t byte = e < 2u ? 0u : e - 2u;
        uint32_t out = 0;
        if (e == 255u) {
            byte = 255u;
            bad = 1;
        } else {
            const float inv = __uint_as_float((254u - byte) << 23);
            out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, x[it][0] * inv, x[it][1] * inv,
                                                           1.0f, 0);
            out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, x[it][2] * inv, x[it][3] * inv,
                                                           1.0f, 1);
        }
        if (q0 + it * (kQuantThreads / 8u) < total) { // the same for a block's lanes
            *(uint16_t *)(codes + row[it] * ld_codes + blk[it] * 16u + part * 2u) = (uint16_t)out;
            if (part == 0)
                scales[row[it] * ld_scales + blk[it]] = (uint8_t)byte;
        }
    }
    zs::raise_flag(flag, bad);
}

// 16-bit rows: four lanes to a block.
template <class Fmt>
__global__ __launch_bounds__(kQuantThreads) void zs_mx_quantize_kernel(
    const typename Fmt::T *__restrict__ src, uint64_t ld_src, uint64_t rows, uint64_t cols,
    uint64_t nb, uint8_t *__restrict__ codes, uint64_t ld_codes, uint8_t *__restrict__ scales,
    uint64_t ld_scales, int32_t *flag) {
    const uint32_t part = threadIdx.x & 3u;
    const uint64_t q0 = (uint64_t)blockIdx.x * kQuantBlocks + threadIdx.x / 4u;
    const uint64_t total = rows * nb;
    int bad = 0;
#pragma unroll
    for (uint32_t it = 0; it < kQuantIters; it++) {
        const uint64_t q = q0 + it * (kQuantThreads / 4u);
        if (q >= total) // the same for the four lanes of a block
            break;
        uint64_t row, blk;
        split_block(q, rows, nb, row, blk);
        const uint64_t c = blk * 32u + part * 8u;
        const typename Fmt::V8 h = load8<Fmt>(src + row * ld_src + c, (int64_t)(cols - c));
        float v[8];
        for (int i = 0; i < 8; i++)
            v[i] = (float)h[i];
        uint32_t amax = 0;
        for (int i = 0; i < 8; i++) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            amax = b > amax ? b : amax;
        }
        amax = quad_max(amax);
        const uint32_t e = amax >> 23;
        uint32_t byte = e < 2u ? 0u : e - 2u;
        uint32_t out = 0;
        if (e == 255u) {
            byte = 255u;
            bad = 1;
        } else {
            const float inv = __uint_as_float((254u - byte) << 23);
            out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0] * inv, v[1] * inv, 1.0f, 0);
            out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2] * inv, v[3] * inv, 1.0f, 1);
            out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4] * inv, v[5] * inv, 1.0f, 2);
            out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6] * inv, v[7] * inv, 1.0f, 3);
        }
        *(uint32_t *)(codes + row * ld_codes + blk * 16u + part * 4u) = out;
        if (part == 0)
            scales[row * ld_scales + blk] = (uint8_t)byte;
    }
    zs::raise_flag(flag, bad);
}

// ---------------------------------------------------------------------------
// Values of one matrix, or of nd flat shards one after the other.
// ---------------------------------------------------------------------------
constexpr uint32_t kMaxShardsPerLaunch = 128; // two pointers each: 2 KiB of arguments

struct ShardArgs {
    const uint8_t *codes[kMaxShardsPerLaunch];
    const uint8_t *scales[kMaxShardsPerLaunch];
};

template <class Fmt>
__global__ __launch_bounds__(kQuantThreads) void zs_mx_dequantize_kernel(
    ShardArgs a, uint64_t rows, uint64_t cols, uint64_t nb, uint64_t ld_codes,
    uint64_t ld_scales, typename Fmt::T *__restrict__ out, uint64_t ld_out,
    uint64_t shard_stride) {
    const uint8_t *codes = a.codes[blockIdx.y];
    const uint8_t *scales = a.scales[blockIdx.y];
    out += (uint64_t)blockIdx.y * shard_stride;
    const uint32_t part = threadIdx.x & 3u;
    const uint64_t q0 = (uint64_t)blockIdx.x * kQuantBlocks + threadIdx.x / 4u;
    const uint64_t total = rows * nb;
#pragma unroll
    for (uint32_t it = 0; it < kQuantIters; it++) {
        const uint64_t q = q0 + it * (kQuantThreads / 4u);
        if (q >= total)
            break;
        uint64_t row, blk;
        split_block(q, rows, nb, row, blk);
        const uint64_t c = blk * 32u + part * 8u;
        const uint32_t code = *(const uint32_t *)(codes + row * ld_codes + blk * 16u + part * 4u);
        const float s = scale_f32(scales[row * ld_scales + blk]);
        // e2m1 to fp32 is exact, and so is the power of two
        const f32x2 d0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 0);
        const f32x2 d1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 1);
        const f32x2 d2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 2);
        const f32x2 d3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code, 1.0f, 3);
        const float v[8] = {d0[0] * s, d0[1] * s, d1[0] * s, d1[1] * s,
                            d2[0] * s, d2[1] * s, d3[0] * s, d3[1] * s};
        typename Fmt::T *o = out + row * ld_out + c;
        if (c + 8 <= cols) {
            if constexpr (sizeof(typename Fmt::T) == 4) {
                *(f32x4_a4 *)o = f32x4{v[0], v[1], v[2], v[3]};
                *(f32x4_a4 *)(o + 4) = f32x4{v[4], v[5], v[6], v[7]};
            } else {
                typename Fmt::V8 h;
                for (int i = 0; i < 8; i++)
                    h[i] = (typename Fmt::T)v[i];
                __builtin_nontemporal_store(__builtin_bit_cast(u32x4, h), (u32x4_a2 *)o);
            }
        } else {
            for (int i = 0; i < 8; i++)
                if (c + i < cols)
                    o[i] = (typename Fmt::T)v[i];
        }
    }
}

template <int V>
struct Const {
    static constexpr int value = V;
};

// ---------------------------------------------------------------------------
// Products with the weight's rows along the output: y[m][n] = sum_k a w.
// For up to kSkinnyM rows of the left operand: one workgroup computes 16
// output columns (16 rows of w), its waves share out K and join in shared
// memory.
// A wave's step is 128 of K: lane l holds row l % 16 and the block l / 16 of
// the step, 16 bytes of codes and one scale.  These kernels take what the one
// that keeps its left operand in registers (below) does not: 33 to 64 rows, K
// past its registers, less than eight blocks.  Bound by the loads of the left
// operand: 64 x 4096 x 4096 in bfloat16 19 us.
// ---------------------------------------------------------------------------
struct MxArgs {
    const uint8_t *codes;
    const uint8_t *scales;
    uint64_t ld_codes, ld_scales;
};

// Sum the waves' partial tiles in order and store them.  acc of wave w: D
// tiles of 16 (n) x 16 (m), register i of lane l at n = 4 (l / 16) + i,
// m = l % 16.
template <int MT>
__device__ __forceinline__ void skinny_join(f32x4 (&acc)[MT], f32x4 *lds, uint64_t n0, uint64_t M,
                                            uint64_t N, void *y, int y_type, uint64_t ld_y) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    for (int t = 0; t < MT; t++)
        lds[(wave * MT + t) * 64 + lane] = acc[t];
    __syncthreads();
    for (uint32_t t = wave; t < MT; t += kSkinnyWaves) {
        f32x4 s = lds[t * 64 + lane];
        for (uint32_t w = 1; w < kSkinnyWaves; w++) {
            const f32x4 p = lds[(w * MT + t) * 64 + lane];
            for (int i = 0; i < 4; i++)
                s[i] += p[i];
        }
        const uint64_t m = t * 16 + (lane & 15u), n = n0 + 4u * (lane >> 4);
        if (m < M && n < N)
            by_type(y_type, [&](auto *o) {
                store4((decltype(o))y + m * ld_y + n, s, (int64_t)(N - n));
            });
    }
}

// The first of this workgroup's 16 columns: a launch has at most kSkinnyGridX
// workgroups along x (HIP counts a dimension's threads in 32 bits), the rest along y.
constexpr uint64_t kSkinnyGridX = 1ull << 22;
__device__ __forceinline__ uint64_t skinny_columns() {
    return ((uint64_t)blockIdx.y * kSkinnyGridX + blockIdx.x) * 16u;
}

// This wave's share of the steps.
__device__ __forceinline__ uint32_t skinny_first(uint32_t steps, uint32_t wave) {
    return steps * wave / kSkinnyWaves;
}

// Blocks past the last one repeat it with scales of 2^-127 on both sides,
// which makes their products 0 (see MxCodes).
template <int MT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void zs_mx_matmul_skinny_kernel(
    MxArgs a, MxArgs w, uint64_t M, uint64_t N, uint32_t nb, void *y, int y_type,
    uint64_t ld_y) {
    __shared__ f32x4 lds[kSkinnyWaves * MT * 64];
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t n0 = skinny_columns(), n = n0 + r < N ? n0 + r : N - 1;
    if (n0 >= N)
        return;
    const uint8_t *wc = w.codes + n * w.ld_codes, *ws = w.scales + n * w.ld_scales;
    f32x4 acc[MT];
    const uint8_t *ac[MT], *as[MT];
    for (int t = 0; t < MT; t++) {
        const uint64_t m = t * 16 + r < M ? t * 16 + r : M - 1;
        ac[t] = a.codes + m * a.ld_codes;
        as[t] = a.scales + m * a.ld_scales;
        acc[t] = f32x4{0, 0, 0, 0};
    }
    const uint32_t steps = (nb + 3) / 4, end = skinny_first(steps, wave + 1);
#pragma unroll 1
    for (uint32_t s = skinny_first(steps, wave); s < end; s++) {
        const bool in = 4 * s + g < nb;
        const uint32_t blk = in ? 4 * s + g : nb - 1;
        const u32x4 c = *(const u32x4 *)(wc + blk * 16u);
        const int cs = in ? ws[blk] : 0;
        const i32x8 vw = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
        for (int t = 0; t < MT; t++) {
            const u32x4 x = *(const u32x4 *)(ac[t] + blk * 16u);
            const int xs = in ? as[t][blk] : 0;
            const i32x8 va = {(int)x[0], (int)x[1], (int)x[2], (int)x[3], 0, 0, 0, 0};
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vw, va, acc[t], 4, 4, 0, cs,
                                                                      0, xs);
        }
    }
    skinny_join<MT>(acc, lds, n0, M, N, y, y_type, ld_y);
}

// x as two bfloat16 pieces whose sum is x exactly: an fp16 value has 11
// significant bits, bfloat16 eight, and the remainder at most three, within
// bfloat16's exponent range.
__device__ __forceinline__ void split_f16(const f16x8 &x, bf16x8 &hi, bf16x8 &lo) {
    for (int i = 0; i < 8; i++) {
        const float f = (float)x[i];
        // truncation keeps the remainder finite and exact (infinities and
        // NaN stay in hi and leave a zero remainder)
        const float h = __uint_as_float(__float_as_uint(f) & 0xFFFF0000u);
        hi[i] = (__bf16)h;
        const float d = f - h;
        lo[i] = (__bf16)((__float_as_uint(f) & 0x7F800000u) == 0x7F800000u ? 0.0f : d);
    }
}

// Eight codes (one dword) as bfloat16 values times 2^(byte - 127): two
// significant bits, exact below 2^128 (from there on, which only the bytes 253
// and 254 reach, infinite).
__device__ __forceinline__ bf16x8 decode8_bf16(uint32_t code, float s) {
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, s, 3);
    return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Eight codes as fp16 values times 2^(byte - 127): exact where fp16 holds
// them (see fits_f16).
__device__ __forceinline__ f16x8 decode8_f16(uint32_t code, float s) {
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, s, 0);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, s, 1);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, s, 2);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code, s, 3);
    return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <class Fmt>
__device__ __forceinline__ typename Fmt::V8 decode8(uint32_t code, float s) {
    if constexpr (Fmt::kType == ZERO_F16)
        return decode8_f16(code, s);
    else
        return decode8_bf16(code, s);
}

// Whether a block's values are fp16 numbers as they are: 0.5 2^e >= 2^-24
// and 6 2^e < 65504 for scale bytes 104 to 140, and a block of zeros.
__device__ __forceinline__ bool fits_f16(uint32_t byte, uint32_t any_code) {
    return byte - 104u <= 36u || (byte != 255u && (any_code & 0x77777777u) == 0);
}

__device__ __forceinline__ f32x4 mfma16(const f16x8 &a, const f16x8 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(const bf16x8 &a, const bf16x8 &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// MFMA j of a step takes dword j of each lane's block, so that a lane's 16
// bytes of codes are one load: its K index 8 g + i stands for the step's
// column 32 g + 8 j + i, for both operands.
template <class Fmt, int MT>
__global__ __launch_bounds__(kSkinnyWaves * 64) void zs_mx_linear_skinny_kernel(
    const typename Fmt::T *__restrict__ x, uint64_t ld_x, MxArgs w, uint64_t M, uint64_t N,
    uint32_t K, uint32_t nb, void *y, int y_type, uint64_t ld_y) {
    __shared__ f32x4 lds[kSkinnyWaves * MT * 64];
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint64_t n0 = skinny_columns(), n = n0 + r < N ? n0 + r : N - 1;
    if (n0 >= N)
        return;
    const uint8_t *wc = w.codes + n * w.ld_codes, *ws = w.scales + n * w.ld_scales;
    f32x4 acc[MT];
    const typename Fmt::T *xr[MT];
    for (int t = 0; t < MT; t++) {
        xr[t] = x + (t * 16 + r < M ? t * 16 + r : M - 1) * ld_x;
        acc[t] = f32x4{0, 0, 0, 0};
    }
    // whole: the step lies inside K (else zeros past the end)
    auto step = [&](auto whole, uint32_t s) {
        const bool in = whole.value || 4 * s + g < nb;
        const uint32_t blk = in ? 4 * s + g : nb - 1, k = 128 * s + 32 * g;
        u32x4 c = *(const u32x4 *)(wc + blk * 16u);
        uint32_t byte = ws[blk];
        typename Fmt::V8 xf[MT][4];
        for (int t = 0; t < MT; t++)
            for (int j = 0; j < 4; j++)
                xf[t][j] = load8<Fmt>(xr[t] + k + 8 * j,
                                      whole.value ? 8 : (int64_t)K - (int64_t)(k + 8 * j));
        if (!in) {
            c = u32x4{0, 0, 0, 0};
            byte = 127;
        }
        const float sc = __uint_as_float(byte << 23);
        if (Fmt::kType != ZERO_F16 || __all(fits_f16(byte, c[0] | c[1] | c[2] | c[3]))) {
            for (int j = 0; j < 4; j++) {
                const typename Fmt::V8 wf = decode8<Fmt>(c[j], sc);
                for (int t = 0; t < MT; t++)
                    acc[t] = mfma16(wf, xf[t][j], acc[t]);
            }
        } else if constexpr (Fmt::kType == ZERO_F16) {
            for (int j = 0; j < 4; j++) {
                const bf16x8 wf = decode8_bf16(c[j], sc);
                for (int t = 0; t < MT; t++) {
                    bf16x8 hi, lo;
                    split_f16(xf[t][j], hi, lo);
                    acc[t] = mfma16(wf, lo, acc[t]);
                    acc[t] = mfma16(wf, hi, acc[t]);
                }
            }
        }
    };
    const uint32_t steps = (nb + 3) / 4, end = skinny_first(steps, wave + 1);
    const uint32_t whole = K / 128u < end ? K / 128u : end;
    uint32_t s = skinny_first(steps, wave);
#pragma unroll 1
    for (; s < whole; s++)
        step(Const<1>(), s);
    if (s < end)
        step(Const<0>(), s);
    skinny_join<MT>(acc, lds, n0, M, N, y, y_type, ld_y);
}

// Up to 32 rows of a left operand short enough that a wave holds its share of
// it in registers (S steps): a workgroup goes over several groups of 16
// output columns, the weight of the next one on its way while one is
// joined.  Only the weight is read in the loop; with the left operand read at
// each step (the kernels above) its loads are four of six.  A pair of steps
// takes its scales from one load of eight bytes a row.  Against the kernels
// above: 5 x 50257 x 1600, bfloat16 17.0 -> 11.9 us (3.7 TB/s), 16 x 32000 x
// 4096 44.6 -> 23.4, 32 x 50257 x 1600 47.2 -> 20.9, 16 x 32000 x 8192 88.5 ->
// 51.7, 4 by 4 bits 1 x 11008 x 4096 10.4 -> 8.2, 1 x 32000 x 4096 20.1 -> 15.1
// (4.6 TB/s).  Where the columns make one round it is the same within 5% (32 x
// 6400 x 1600 10.1 us against 10.6).  Loading the next group a whole group
// earlier costs more registers than it gains (8.2 -> 11.2).
template <class Fmt, int S_, int MT_>
struct LeftRows {
    typedef typename Fmt::T T;
    static constexpr int S = S_, MT = MT_; // steps; tiles of 16 rows
    static constexpr bool kChecks = Fmt::kType == ZERO_F16; // the weight's range
    typename Fmt::V8 x[MT][S][4];
    const T *row[MT];
    uint32_t k0, K;

    __device__ __forceinline__ void load(const T *p, uint64_t ld, MxArgs, uint64_t M, uint32_t K_,
                                         uint32_t, uint32_t first, uint32_t count) {
        const uint32_t r = threadIdx.x & 15u, g = threadIdx.x >> 4 & 3u;
        K = K_;
        k0 = 128u * first + 32u * g;
#pragma unroll
        for (uint32_t t = 0; t < MT; t++) {
            row[t] = p + (16 * t + r < M ? 16 * t + r : M - 1) * ld;
#pragma unroll
            for (uint32_t i = 0; i < S; i++) {
                const uint32_t k = k0 + 128u * i;
#pragma unroll
                for (uint32_t j = 0; j < 4; j++)
                    x[t][i][j] = typename Fmt::V8{};
                if (128u * (first + i + 1) <= K) {
                    if (i < count)
#pragma unroll
                        for (uint32_t j = 0; j < 4; j++)
                            x[t][i][j] = load8<Fmt>(row[t] + k + 8 * j, 8);
                } else if (i < count) {
#pragma unroll
                    for (uint32_t j = 0; j < 4; j++)
                        x[t][i][j] =
                            load8<Fmt>(row[t] + k + 8 * j, (int64_t)K - (int64_t)(k + 8 * j));
                }
            }
        }
    }
    __device__ __forceinline__ void multiply(f32x4 (&acc)[MT], int i, const u32x4 &c,
                                             uint32_t b) const {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const typename Fmt::V8 wf = decode8<Fmt>(c[j], __uint_as_float(b << 23));
#pragma unroll
            for (int t = 0; t < MT; t++)
                acc[t] = mfma16(wf, x[t][i][j], acc[t]);
        }
    }
    // the same for any scales (see split_f16), from memory
    __device__ __forceinline__ void exact(f32x4 (&acc)[MT], const uint8_t *codes,
                                          const uint8_t *scales, uint32_t nb,
                                          uint32_t count) const {
        if constexpr (Fmt::kType == ZERO_F16) {
#pragma unroll 1
            for (uint32_t i = 0; i < 4 * count; i++) {
                const uint32_t k = k0 + 128u * (i / 4) + 8u * (i % 4);
                uint32_t code = 0, byte = 127;
                if (k / 32u < nb) {
                    code = *(const uint32_t *)(codes + k / 32u * 16u + 4u * (i % 4));
                    byte = scales[k / 32u];
                }
                const bf16x8 wf = decode8_bf16(code, __uint_as_float(byte << 23));
#pragma unroll
                for (int t = 0; t < MT; t++) {
                    bf16x8 hi, lo;
                    split_f16(load8<Fmt>(row[t] + k, (int64_t)K - (int64_t)k), hi, lo);
                    acc[t] = mfma16(wf, lo, acc[t]);
                    acc[t] = mfma16(wf, hi, acc[t]);
                }
            }
        }
    }
};

template <int S_, int MT_>
struct LeftMx {
    typedef uint8_t T;
    static constexpr int S = S_, MT = MT_;
    static constexpr bool kChecks = false;
    u32x4 x[MT][S];
    uint32_t byte[MT][S];

    // blocks past the last one are zeros
    __device__ __forceinline__ void load(const T *, uint64_t, MxArgs a, uint64_t M, uint32_t,
                                         uint32_t nb, uint32_t first, uint32_t count) {
        const uint32_t r = threadIdx.x & 15u, g = threadIdx.x >> 4 & 3u;
#pragma unroll
        for (uint32_t t = 0; t < MT; t++) {
            const uint64_t m = 16 * t + r < M ? 16 * t + r : M - 1;
#pragma unroll
            for (uint32_t i = 0; i < S; i++) {
                const uint32_t blk = 4u * (first + i) + g;
                x[t][i] = u32x4{0, 0, 0, 0};
                byte[t][i] = 127;
                if (i < count && blk < nb) {
                    x[t][i] = *(const u32x4 *)(a.codes + m * a.ld_codes + blk * 16u);
                    byte[t][i] = a.scales[m * a.ld_scales + blk];
                }
            }
        }
    }
    __device__ __forceinline__ void exact(f32x4 (&)[MT], const uint8_t *, const uint8_t *,
                                          uint32_t, uint32_t) const {}
    __device__ __forceinline__ void multiply(f32x4 (&acc)[MT], int i, const u32x4 &c,
                                             uint32_t b) const {
        const i32x8 vw = {(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < MT; t++) {
            const u32x4 &v = x[t][i];
            const i32x8 va = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
            acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(vw, va, acc[t], 4, 4, 0,
                                                                      (int)b, 0, (int)byte[t][i]);
        }
    }
};

// nb >= 8.  A lane's block past the last one repeats that one's codes with a
// scale of 2^-127, which keeps them finite, against zeros of the left operand.
template <class Left, int OCC>
__global__ __launch_bounds__(kSkinnyWaves * 64, OCC) void zs_mx_rows_kernel(
    const typename Left::T *x, uint64_t ld_x, MxArgs a, MxArgs w, uint64_t M, uint64_t N,
    uint32_t K, uint32_t nb, uint32_t groups, void *y, int y_type, uint64_t ld_y) {
    constexpr int S = Left::S, MT = Left::MT;
    static_assert(S % 2 == 0, "steps take their scales in pairs");
    __shared__ f32x4 lds[2][MT][kSkinnyWaves * 64];
    __shared__ uint32_t outside; // whether a block lay outside fp16
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, g = lane >> 4;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t steps = (nb + 3) / 4, first = skinny_first(steps, wave);
    const uint32_t count = skinny_first(steps, wave + 1) - first;
    constexpr uint32_t kPast = 0x0C0C0C0Cu; // selects a byte of 0
    uint32_t code_at[S], pair_at[S / 2], sel[S];
#pragma unroll
    for (uint32_t i = 0; i < S; i++) {
        const uint32_t blk = 4u * (first + i) + g;
        code_at[i] = (blk < nb ? blk : nb - 1) * 16u;
        const uint32_t pair = 4u * (first + (i & ~1u)), p = pair + 8u <= nb ? pair : nb - 8u;
        pair_at[i / 2] = p;
        const uint32_t byte = blk - p;
        sel[i] = blk < nb ? 0x0C0C0C00u | (byte & 7u) : kPast;
    }
    struct Weight {
        u32x4 c[S];
        uint64_t b[S / 2];
    };
    auto row_of = [&](uint32_t group) {
        const uint64_t n = (uint64_t)group * 16u + r;
        return n < N ? n : N - 1;
    };
    auto load = [&](uint32_t group, Weight &d) {
        typedef uint64_t u64_a1 __attribute__((aligned(1)));
        const uint64_t n = row_of(group);
        const uint8_t *codes = w.codes + n * w.ld_codes, *scales = w.scales + n * w.ld_scales;
#pragma unroll
        for (uint32_t i = 0; i < S; i++) {
            if (i % 2 == 0 && i < count)
                d.b[i / 2] = *(const u64_a1 *)(scales + pair_at[i / 2]);
            if (i < count)
                d.c[i] = *(const u32x4 *)(codes + code_at[i]);
        }
    };
    Left left;
    Weight now;
    uint32_t buf = 0;
    // the waves' parts of a group of columns, summed and stored
    auto join = [&](const f32x4 (&acc)[MT], uint64_t n0) {
#pragma unroll
        for (int t = 0; t < MT; t++)
            lds[buf & 1][t][wave * 64 + lane] = acc[t];
        __syncthreads();
        // each wave sums two rows of a tile, half of the waves' parts in
        // either half of its lanes; it is done before it reaches the next
        // barrier, after which this buffer is written again
#pragma unroll
        for (int t = 0; t < MT; t++) {
            if (16u * t + 2u * wave >= M)
                break;
            const uint32_t m = 2u * wave + (lane >> 4 & 1u);
            const float *p = (const float *)lds[buf & 1][t] +
                             ((lane >> 5) * (kSkinnyWaves / 2) * 64u + m + 16u * (r >> 2)) * 4u +
                             (r & 3u);
            float sum = p[0];
#pragma unroll
            for (uint32_t v = 1; v < kSkinnyWaves / 2; v++)
                sum += p[v * 256u];
            sum += __shfl_xor(sum, 32);
            const uint64_t n = n0 + r;
            if (lane < 32 && 16u * t + m < M && n < N)
                by_type(y_type, [&](auto *o) {
                    typedef decltype(o) P;
                    ((P)y)[(16u * t + m) * ld_y + n] =
                        (typename std::remove_pointer<P>::type)sum;
                });
        }
        buf++;
    };
    load(blockIdx.x, now);
    left.load(x, ld_x, a, M, K, nb, first, count);
    if (Left::kChecks) {
        if (threadIdx.x == 0)
            outside = 0;
        __syncthreads();
    }
#pragma unroll 1
    for (uint32_t group = blockIdx.x; group < groups;) {
        f32x4 acc[MT] = {};
        bool fits = true;
#pragma unroll
        for (uint32_t i = 0; i < S; i++)
            if (i < count) {
                const uint32_t byte = __builtin_amdgcn_perm((uint32_t)(now.b[i / 2] >> 32),
                                                            (uint32_t)now.b[i / 2], sel[i]);
                if (Left::kChecks)
                    fits &= sel[i] == kPast ||
                            fits_f16(byte, now.c[i][0] | now.c[i][1] | now.c[i][2] | now.c[i][3]);
                left.multiply(acc, i, now.c[i], byte);
            }
        if (Left::kChecks && !fits)
            outside = 1;
        // the next group's weight comes while this one is joined
        const uint64_t n0 = (uint64_t)group * 16u;
        group += gridDim.x;
        if (group < groups)
            load(group, now);
        join(acc, n0);
    }
    // fp16 that met a block outside its range: all of this workgroup's
    // columns again (5 x 50257 x 1600 with one such block 13 -> 36 us, with one
    // in every row 53)
    if (Left::kChecks && __builtin_amdgcn_readfirstlane(outside) != 0) {
#pragma unroll 1
        for (uint32_t group = blockIdx.x; group < groups; group += gridDim.x) {
            f32x4 acc[MT] = {};
            const uint64_t n = row_of(group);
            left.exact(acc, w.codes + n * w.ld_codes, w.scales + n * w.ld_scales, nb, count);
            join(acc, (uint64_t)group * 16u);
        }
    }
}

// ---------------------------------------------------------------------------
// Tiled products.  A workgroup of eight waves, two along m and four along
// the output's columns, computes a tile of 32 FM rows and 64 FN columns; a
// wave holds FM x FN tiles of 16 x 16 in registers.  The inner dimension
// advances by one 128-byte row of shared memory per operand: 256 codes, or
// 64 values of 16 bits.  Two such steps fit: while one is computed the next
// one's loads are in flight, and one barrier ends a step.  Within a step the
// left operand's fragments stream through four registers, three ahead of
// the MFMAs, and the weight's second half is read during the first.
// The 16-byte chunk c of row r lies in slot c ^ f(r), so that the rows a
// fragment's lanes read, in either order below, fall into different banks.
// Bound by the reads of shared memory between the matrix instructions (the
// matrix cores are busy 43-47% of the time).  8192 x 11008 x 4096 in 4 bits 224
// us (3.3 PF/s), fp16 activations 2047 x 6400 x 1600 48 us (0.87 PF/s, 200
// tiles on 256 CUs), the gradient 4096 x 4096 x 11008 372 us (0.99 PF/s).
// ---------------------------------------------------------------------------
constexpr uint32_t kTileThreads = 512;
constexpr uint32_t kStepBytes = 128; // of a row, per step

__device__ __forceinline__ uint32_t chunk_of(uint32_t row, uint32_t slot) {
    return slot ^ ((row ^ row >> 3) & 7u);
}
__device__ __forceinline__ uint32_t chunk_at(uint32_t row, uint32_t chunk) {
    return row * kStepBytes + chunk_of(row, chunk) * 16u;
}

// The tile of workgroup `id`: each of the eight XCDs (consecutive workgroups
// go round them) takes a run of consecutive tiles, and tiles go in groups of
// eight along m so that neighbours share rows of both operands in L2.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tm, uint32_t tn, uint32_t &im,
                                        uint32_t &in) {
    const uint32_t total = tm * tn, run = total / 8u, rest = total % 8u;
    const uint32_t xcd = id % 8u, at = id / 8u;
    const uint32_t t = xcd * run + (xcd < rest ? xcd : rest) + at;
    const uint32_t group = t / (8u * tn), first = group * 8u;
    const uint32_t rows = tm - first < 8u ? tm - first : 8u;
    const uint32_t in_group = t - group * 8u * tn;
    im = first + in_group % rows;
    in = in_group / rows;
}

// The matrix cores get the weight as the first operand, so that a lane ends
// up with four consecutive columns of y in a tile of 16 x 16.  Where a wave
// has pairs of tiles, row 4 g + i of tile t stands for column 32 (t / 2) + 8 g
// + 4 (t % 2) + i of the wave's: two tiles then give a lane eight columns, and
// a store of 64 lanes fills 64 bytes of each of its rows.
template <int FN>
__device__ __forceinline__ uint32_t weight_row(uint32_t t, uint32_t r) {
    return FN % 2 == 0 ? t / 2u * 32u + (r >> 2) * 8u + t % 2u * 4u + (r & 3u) : t * 16u + r;
}

// Store up to eight consecutive fp32 results.
template <class T>
__device__ __forceinline__ void store8(T *y, const f32x4 &a, const f32x4 &b, int64_t valid) {
    if constexpr (sizeof(T) == 2) {
        typedef T T8 __attribute__((ext_vector_type(8)));
        if (valid >= 8) { // nontemporal: 8192 x 11008 x 4096 in 4 bits 235 -> 225 us
            const T8 v = {(T)a[0], (T)a[1], (T)a[2], (T)a[3],
                          (T)b[0], (T)b[1], (T)b[2], (T)b[3]};
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), (u32x4_a2 *)y);
            return;
        }
    }
    store4(y, a, valid);
    store4(y + 4, b, valid - 4);
}

// Store a wave's tiles.
template <int FM, int FN>
__device__ __forceinline__ void store_tiles(const f32x4 (&acc)[FN][FM], uint64_t m0, uint64_t n0,
                                            uint64_t M, uint64_t N, void *y, int y_type,
                                            uint64_t ld_y) {
    const uint32_t lane = threadIdx.x & 63u;
    m0 += lane & 15u;
    n0 += (FN % 2 == 0 ? 8u : 4u) * (lane >> 4);
    by_type(y_type, [&](auto *t) {
#pragma unroll
        for (int j = 0; j < FM; j++) {
            const uint64_t m = m0 + j * 16;
            decltype(t) row = (decltype(t))y + m * ld_y;
            if constexpr (FN % 2 == 0) {
#pragma unroll
                for (int p = 0; p < FN / 2; p++) {
                    const uint64_t n = n0 + p * 32;
                    if (m < M && n < N)
                        store8(row + n, acc[2 * p][j], acc[2 * p + 1][j], (int64_t)(N - n));
                }
            } else {
#pragma unroll
                for (int i = 0; i < FN; i++) {
                    const uint64_t n = n0 + i * 16;
                    if (m < M && n < N)
                        store4(row + n, acc[i][j], (int64_t)(N - n));
                }
            }
        }
    });
}

// Where a wave's fragments lie in a buffer.  16 rows on, the swizzle differs
// by a constant: bits 1 and 2 of the slot, by twice the distance (a wave's
// first row is a multiple of 16 times its tiles, so nothing is carried).
template <int FN>
struct FragAt {
    uint32_t left[2], weight[2][2];

    __device__ __forceinline__ void init(uint32_t left_row, uint32_t weight_row0) {
        const uint32_t r = threadIdx.x & 15u, g = threadIdx.x >> 4 & 3u;
        for (uint32_t ks = 0; ks < 2; ks++) {
            left[ks] = chunk_at(left_row + r, ks * 4 + g);
            for (uint32_t t = 0; t < 2; t++)
                weight[ks][t] = chunk_at(weight_row0 + weight_row<FN>(t, r), ks * 4 + g);
        }
    }
    // j: in rows of 16
    __device__ __forceinline__ static u32x4 read(const uint8_t *buf, uint32_t at, uint32_t j) {
        return *(const u32x4 *)(buf + (at ^ (2u * j & 6u) * 16u) + j * 2048u);
    }
    __device__ __forceinline__ u32x4 read_left(const uint8_t *buf, uint32_t ks,
                                               uint32_t j) const {
        return read(buf, left[ks], j);
    }
    __device__ __forceinline__ u32x4 read_weight(const uint8_t *buf, uint32_t ks,
                                                 uint32_t t) const {
        return FN % 2 == 0 ? read(buf, weight[ks][t % 2u], t / 2u * 2u)
                           : read(buf, weight[ks][0], t);
    }
};

// The MFMAs of a step from a buffer, `between` called once the first
// fragments are on their way.
template <int FM, int FN, class Mfma, class Between>
__device__ __forceinline__ void run_step(const FragAt<FN> &at, const uint8_t *buf, Mfma mfma,
                                         Between between) {
    u32x4 w0[FN], w1[FN], x[4];
#pragma unroll
    for (uint32_t i = 0; i < FN; i++)
        w0[i] = at.read_weight(buf, 0, i);
#pragma unroll
    for (uint32_t j = 0; j < 3 && j < 2 * FM; j++)
        x[j] = at.read_left(buf, j / FM, j % FM);
    between();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (uint32_t j = 0; j < 2 * FM; j++) {
        if (j + 3 < 2 * FM)
            x[(j + 3) % 4] = at.read_left(buf, (j + 3) / FM, (j + 3) % FM);
        // a share of the second half's weight, all of it by the half's end
        if (j < FM)
#pragma unroll
            for (uint32_t i = j * FN / FM; i < (j + 1) * FN / FM; i++)
                w1[i] = at.read_weight(buf, 1, i);
#pragma unroll
        for (uint32_t i = 0; i < FN; i++) {
            if (j < FM)
                mfma(Const<0>(), i, j, w0[i], x[j % 4]);
            else
                mfma(Const<1>(), i, j - FM, w1[i], x[j % 4]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// 16 bytes for each lane of this wave from base + off straight into shared
// memory at lds_at + 16 * lane.  The compiler does not count these loads:
// dma_wait before the barrier that publishes them.  m0 is reserved (naming it
// as clobbered is warned of): the compiler sets it right before what needs it,
// which in these kernels is nothing but this.
__device__ __forceinline__ void dma16(uint32_t lds_at, const void *base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(
                     lds_at),
                 "v"(off), "s"(base)
                 : "memory");
}
__device__ __forceinline__ void dma_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_address(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// The codes of one operand of the 4-bit product: a tile of ROWS rows, copied
// to shared memory in pieces of 64.  Rows past the matrix repeat its last
// one (their results are dropped) and blocks past the last repeat that one
// (their scales are 2^-127 on both sides, which makes each product with them
// 0: at most 36 * 2^-254, far below fp32's smallest).
template <uint32_t ROWS>
struct MxCodes {
    static constexpr uint32_t kPieces = ROWS / 64u;
    const uint8_t *base;
    uint32_t off[kPieces], chunk;

    __device__ __forceinline__ void init(const MxArgs &q, uint64_t row0, uint64_t rows) {
        base = q.codes + row0 * q.ld_codes;
        const uint32_t last = rows - 1 - row0 < ROWS ? (uint32_t)(rows - 1 - row0) : ROWS - 1;
        const uint32_t r0 = threadIdx.x / 8u;
        chunk = chunk_of(r0, threadIdx.x % 8u); // rows 64 apart swizzle alike
        for (uint32_t j = 0; j < kPieces; j++) {
            const uint32_t r = r0 + 64u * j;
            off[j] = (r < last ? r : last) * (uint32_t)q.ld_codes + chunk * 16u;
        }
    }
    // the step from block blk0 on, to this wave's place `to` of the buffer
    __device__ __forceinline__ void copy(uint64_t nb, uint64_t blk0, uint32_t to) const {
        const uint32_t back =
            blk0 + chunk < nb ? 0u : (uint32_t)(blk0 + chunk - (nb - 1)) * 16u;
#pragma unroll
        for (uint32_t j = 0; j < kPieces; j++)
            dma16(to + j * 64u * kStepBytes, base + blk0 * 16u, off[j] - back);
    }
};

// Both operands in 4 bits, copied straight to shared memory.
template <int FM, int FN>
__global__ __launch_bounds__(kTileThreads, 2) void zs_mx_matmul_tile_kernel(
    MxArgs a, MxArgs w, uint64_t M, uint64_t N, uint64_t nb, uint32_t tm, uint32_t tn, void *y,
    int y_type, uint64_t ld_y) {
    constexpr uint32_t TM = 32 * FM, TN = 64 * FN, kBytes = (TM + TN) * kStepBytes;
    static_assert(TM + TN <= kTileThreads, "a thread loads a row's scales");
    __shared__ __align__(16) uint8_t codes[2][kBytes];
    __shared__ uint2 scales[2][kTileThreads];
    uint32_t im, in;
    tile_of(blockIdx.x, tm, tn, im, in);
    const uint64_t m0 = (uint64_t)im * TM, n0 = (uint64_t)in * TN;
    const uint32_t t = threadIdx.x, lane = t & 63u, wave = t >> 6;
    const uint32_t r = lane & 15u, g = lane >> 4;
    const uint32_t wm = (wave & 1u) * (16 * FM), wn = (wave >> 1) * (16 * FN);
    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FM; j++)
            acc[i][j] = f32x4{0, 0, 0, 0};
    MxCodes<TM> ca;
    MxCodes<TN> cw;
    ca.init(a, m0, M);
    cw.init(w, n0, N);
    FragAt<FN> at;
    at.init(wm, TM + wn);
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds_address(codes) + (t & ~63u) * 16u);
    // this thread's row of scales; threads past the tile's rows repeat one
    const uint64_t rm = m0 + t < M ? m0 + t : M - 1;
    const uint64_t rn = n0 + t - TM < N ? n0 + t - TM : N - 1;
    const uint8_t *row_scales =
        t < TM ? a.scales + rm * a.ld_scales : w.scales + rn * w.ld_scales;
    uint64_t sc = 0;
    const uint64_t steps = (nb + 7) / 8;
    // The eight bytes of a step, 0 past the last block; without a branch once
    // there are eight blocks in all, so that a step's code stays one block.
    auto load = [&](uint64_t s) {
        typedef uint64_t u64_a1 __attribute__((aligned(1)));
        const uint64_t p = 8 * s + 8 <= nb ? 8 * s : nb - 8;
        sc = *(const u64_a1 *)(row_scales + p); // shifted when it is stored: it is waited for there
    };
    auto copy = [&](uint64_t s) {
        const uint32_t lds = to + (uint32_t)(s & 1) * kBytes;
        ca.copy(nb, 8 * s, lds);
        cw.copy(nb, 8 * s, lds + TM * kStepBytes);
    };
    // as four pairs: block g and block 4 + g of the step, the two bytes a
    // lane's MFMAs select
    auto store_scales = [&](uint64_t s) {
        const uint64_t v = 8 * s + 8 <= nb || nb < 8 ? sc : sc >> (8 * (8 * s + 8 - nb));
        scales[s & 1][t] =
            uint2{__builtin_amdgcn_perm((uint32_t)(v >> 32), (uint32_t)v, 0x05010400u),
                  __builtin_amdgcn_perm((uint32_t)(v >> 32), (uint32_t)v, 0x07030602u)};
    };
    auto step = [&](uint64_t s, auto more) {
        uint32_t xa[FM], xw[FN];
        const uint16_t *p = (const uint16_t *)scales[s & 1] + g;
#pragma unroll
        for (uint32_t i = 0; i < FN; i++)
            xw[i] = p[(TM + wn + weight_row<FN>(i, r)) * 4];
#pragma unroll
        for (uint32_t j = 0; j < FM; j++)
            xa[j] = p[(wm + j * 16 + r) * 4];
        run_step<FM, FN>(
            at, codes[s & 1],
            [&](auto ks, uint32_t i, uint32_t j, const u32x4 &fw, const u32x4 &fa) {
                const i32x8 vw = {(int)fw[0], (int)fw[1], (int)fw[2], (int)fw[3], 0, 0, 0, 0};
                const i32x8 va = {(int)fa[0], (int)fa[1], (int)fa[2], (int)fa[3], 0, 0, 0, 0};
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    vw, va, acc[i][j], 4, 4, ks.value, (int)xw[i], ks.value, (int)xa[j]);
            },
            [&]() {
                if constexpr (more.value != 0) {
                    load(s + 1);
                    copy(s + 1);
                }
            });
        if constexpr (more.value != 0) {
            store_scales(s + 1);
            dma_wait();
            __syncthreads();
        }
    };
    if (nb >= 8)
        load(0);
    else
        for (uint64_t b = nb; b > 0; b--)
            sc = sc << 8 | row_scales[b - 1];
    copy(0);
    store_scales(0);
    dma_wait();
    __syncthreads();
#pragma unroll 1
    for (uint64_t s = 0; s + 1 < steps; s++)
        step(s, Const<1>());
    step(steps - 1, Const<0>());
    store_tiles<FM, FN>(acc, m0 + wm, n0 + wn, M, N, y, y_type, ld_y);
}

// This thread's chunks of a tile of ROWS rows of 16-bit values, 64 a step;
// values past `inner` are zero, rows past the matrix repeat its last one.
template <class Fmt, uint32_t ROWS>
struct HalfStage {
    static constexpr uint32_t kChunks = ROWS * 8u / kTileThreads;
    const typename Fmt::T *base;
    uint32_t off[kChunks]; // from the tile's first row
    struct Data {
        typename Fmt::V8 c[kChunks];
    };

    __device__ __forceinline__ void init(const typename Fmt::T *x, uint64_t ld, uint64_t row0,
                                         uint64_t rows) {
        base = x + row0 * ld;
        const uint32_t last = rows - 1 - row0 < ROWS ? (uint32_t)(rows - 1 - row0) : ROWS - 1;
        for (uint32_t j = 0; j < kChunks; j++) {
            const uint32_t r = (j * kTileThreads + threadIdx.x) / 8u;
            off[j] = (r < last ? r : last) * (uint32_t)ld + threadIdx.x % 8u * 8u;
        }
    }
    template <class Whole>
    __device__ __forceinline__ void load(Whole, Data &d, uint64_t inner, uint64_t at) const {
        const int64_t left =
            Whole::value ? 8 : (int64_t)inner - (int64_t)(at + threadIdx.x % 8u * 8u);
#pragma unroll
        for (uint32_t j = 0; j < kChunks; j++)
            d.c[j] = load8<Fmt>(base + at + off[j], left);
    }
    __device__ __forceinline__ void store(const Data &d, uint8_t *lds) const {
#pragma unroll
        for (uint32_t j = 0; j < kChunks; j++) {
            const uint32_t i = j * kTileThreads + threadIdx.x;
            *(typename Fmt::V8 *)(lds + chunk_at(i / 8u, i % 8u)) = d.c[j];
        }
    }
};

// Part `part` of a sum over `inner` rows of w and columns of x, in whole units:
// the operands move to its first row, its results go to fp32 partial sums.
struct Part {
    uint32_t parts;
    float *partial; // parts x M x C

    template <class X>
    __device__ __forceinline__ void take(uint32_t part, uint32_t unit, X &x, MxArgs &w,
                                         uint64_t M, uint64_t C, uint64_t &inner, void *&y,
                                         int &y_type, uint64_t &ld_y) const {
        if (parts == 1)
            return;
        const uint64_t units = (inner + unit - 1) / unit;
        const uint64_t begin = units * part / parts * unit;
        const uint64_t end = units * (part + 1) / parts * unit;
        x += begin;
        w.codes += begin * w.ld_codes;
        w.scales += begin * w.ld_scales;
        inner = (end < inner ? end : inner) - begin;
        y = partial + part * M * C;
        y_type = ZERO_F32;
        ld_y = C;
    }
};

// The parts' sums, in order; a workgroup for 256 columns of a row.
template <class T>
__global__ __launch_bounds__(256) void zs_mx_join_kernel(const float *__restrict__ partial,
                                                         uint32_t parts, uint64_t M, uint64_t C,
                                                         T *__restrict__ y, uint64_t ld_y) {
    const uint64_t c = (uint64_t)blockIdx.x * 256u + threadIdx.x, m = blockIdx.y;
    if (c >= C)
        return;
    const float *p = partial + m * C + c;
    float s = *p;
#pragma unroll 8
    for (uint32_t i = 1; i < parts; i++)
        s += p[i * M * C];
    y[m * ld_y + c] = (T)s;
}

// The weight's side of linear: COLS rows of w, 64 of K a step, decoded to
// the activations' format.  A thread takes a block of 32.
template <class Fmt, uint32_t COLS>
struct RowStage {
    static constexpr uint32_t kBlocks = COLS * 2u; // of a step
    static_assert(kBlocks <= kTileThreads, "a thread takes one block");
    static constexpr bool kSplits = false;
    const uint8_t *codes, *scales;
    uint32_t code_off, scale_off; // from the tile's first row
    struct Data {
        u32x4 c;
        uint32_t byte;
    };

    __device__ __forceinline__ void init(const MxArgs &w, uint64_t n0, uint64_t N) {
        codes = w.codes + n0 * w.ld_codes;
        scales = w.scales + n0 * w.ld_scales;
        const uint32_t last = N - 1 - n0 < COLS ? (uint32_t)(N - 1 - n0) : COLS - 1;
        const uint32_t r = threadIdx.x / 2u < last ? threadIdx.x / 2u : last;
        code_off = r * (uint32_t)w.ld_codes + threadIdx.x % 2u * 16u;
        scale_off = r * (uint32_t)w.ld_scales + threadIdx.x % 2u;
    }
    template <class Whole>
    __device__ __forceinline__ void load(Whole, Data &d, const MxArgs &, uint64_t K,
                                         uint64_t at) const {
        const uint64_t blk = at / 32u;
        if (!Whole::value) {
            d.c = u32x4{0, 0, 0, 0};
            d.byte = 127;
        }
        if (Whole::value || blk + threadIdx.x % 2u < (K + 31) / 32) {
            d.c = *(const u32x4 *)(codes + blk * 16u + code_off);
            d.byte = *(scales + blk + scale_off);
        }
    }
    // false: a value that the format does not hold
    __device__ __forceinline__ bool store(const Data &d, uint8_t *lds) const {
        if (kBlocks < kTileThreads && threadIdx.x >= kBlocks)
            return true;
        const float s = __uint_as_float(d.byte << 23);
#pragma unroll
        for (uint32_t i = 0; i < 4; i++)
            *(typename Fmt::V8 *)(lds +
                                  chunk_at(threadIdx.x / 2u, threadIdx.x % 2u * 4u + i)) =
                decode8<Fmt>(d.c[i], s);
        return Fmt::kType != ZERO_F16 ||
               fits_f16(d.byte, d.c[0] | d.c[1] | d.c[2] | d.c[3]);
    }
    // the same values of row n, eight from k, in bfloat16
    static __device__ __forceinline__ bf16x8 exact8(const MxArgs &w, uint64_t n, uint64_t N,
                                                    uint64_t K, uint64_t k) {
        uint32_t code = 0, byte = 127;
        if (k / 32u < (K + 31) / 32) {
            n = n < N ? n : N - 1;
            code = *(const uint32_t *)(w.codes + n * w.ld_codes + k / 2u);
            byte = w.scales[n * w.ld_scales + k / 32u];
        }
        return decode8_bf16(code, __uint_as_float(byte << 23));
    }
};

// The weight's side of the input's gradient: COLS columns of w, 64 of its
// rows a step, decoded and turned so that a column's values lie together.  A
// thread takes eight columns of four rows, neighbours the next eight, so
// that 32 threads read 128 bytes of a row (with the rows to neighbours the
// gradient of 4096 x 4096 x 11008 took 508 us, now 372).
template <class Fmt, uint32_t COLS>
struct ColumnStage {
    static constexpr uint32_t kAcross = COLS / 8u, kThreads = kAcross * 16u;
    static_assert(kThreads <= kTileThreads, "a thread takes one group");
    static constexpr bool kSplits = true; // see Part
    const uint8_t *codes, *scales;
    uint32_t code_off, scale_off; // of the first of the four rows
    uint32_t ld_codes, ld_scales;
    struct Data {
        uint32_t c[4], byte[4];
    };

    // columns past the matrix repeat its last group (their results are
    // dropped)
    __device__ __forceinline__ void init(const MxArgs &w, uint64_t k0, uint64_t K) {
        const uint64_t last = (K - 1) / 8u * 8u - k0;
        codes = w.codes + k0 / 2u;
        scales = w.scales + k0 / 32u;
        ld_codes = (uint32_t)w.ld_codes;
        ld_scales = (uint32_t)w.ld_scales;
        const uint32_t n = threadIdx.x / kAcross * 4u, k = threadIdx.x % kAcross * 8u;
        const uint32_t at = (uint32_t)(k < last ? k : last);
        code_off = n * ld_codes + at / 2u;
        scale_off = n * ld_scales + at / 32u;
    }
    template <class Whole>
    __device__ __forceinline__ void load(Whole, Data &d, const MxArgs &, uint64_t N,
                                         uint64_t at) const {
        if (kThreads < kTileThreads && threadIdx.x >= kThreads)
            return;
        const uint64_t n = at + threadIdx.x / kAcross * 4u;
#pragma unroll
        for (uint32_t q = 0; q < 4; q++) {
            if (!Whole::value) {
                d.c[q] = 0;
                d.byte[q] = 127;
            }
            if (Whole::value || n + q < N) {
                d.c[q] = *(const uint32_t *)(codes + (at + q) * ld_codes + code_off);
                d.byte[q] = *(scales + (at + q) * ld_scales + scale_off);
            }
        }
    }
    __device__ __forceinline__ bool store(const Data &d, uint8_t *lds) const {
        if (kThreads < kTileThreads && threadIdx.x >= kThreads)
            return true;
        bool ok = true;
        u32x4 v[4];
#pragma unroll
        for (uint32_t q = 0; q < 4; q++) {
            if (Fmt::kType == ZERO_F16)
                ok &= fits_f16(d.byte[q], d.c[q]);
            v[q] = __builtin_bit_cast(u32x4,
                                      decode8<Fmt>(d.c[q], __uint_as_float(d.byte[q] << 23)));
        }
        const uint32_t col = threadIdx.x % kAcross * 8u, n4 = threadIdx.x / kAcross;
#pragma unroll
        for (uint32_t e = 0; e < 8; e++) {
            const uint32_t sel = e % 2u ? 0x07060302u : 0x05040100u, i = e / 2u;
            const uint2 p = {__builtin_amdgcn_perm(v[1][i], v[0][i], sel),
                             __builtin_amdgcn_perm(v[3][i], v[2][i], sel)};
            *(uint2 *)(lds + chunk_at(col + e, n4 / 2u) + (n4 % 2u) * 8u) = p;
        }
        return ok;
    }
    // column k, eight rows from n
    static __device__ __forceinline__ bf16x8 exact8(const MxArgs &w, uint64_t k, uint64_t K,
                                                    uint64_t N, uint64_t n) {
        bf16x8 r;
        for (uint32_t i = 0; i < 8; i++) {
            uint32_t code = 0, byte = 127;
            if (n + i < N && k < K) {
                code = w.codes[(n + i) * w.ld_codes + k / 2u] >> (4 * (k % 2u));
                byte = w.scales[(n + i) * w.ld_scales + k / 32u];
            }
            r[i] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, __uint_as_float(byte << 23),
                                                             0)[0];
        }
        return r;
    }
};

// A wave's tiles of the same product for any scales, from memory: fp16 x in
// two bfloat16 pieces (see split_f16) against the weight in bfloat16.
template <class Stage, int FM, int FN>
__device__ __forceinline__ void exact_tiles(const _Float16 *x, uint64_t ld_x, const MxArgs &w,
                                            uint64_t m0, uint64_t c0, uint64_t M, uint64_t C,
                                            uint64_t I, void *y, int y_type, uint64_t ld_y) {
    const uint32_t lane = threadIdx.x & 63u, r = lane & 15u, g = lane >> 4;
#pragma unroll 1
    for (uint32_t tile = 0; tile < FM * FN; tile++) {
        const uint32_t i = tile / FM, j = tile % FM;
        const uint64_t row = m0 + j * 16 + r, m = row < M ? row : M - 1;
        f32x4 acc = {0, 0, 0, 0};
#pragma unroll 1
        for (uint64_t k = 8 * g; k < I + 8 * g; k += 32) {
            bf16x8 hi, lo;
            split_f16(load8<F16>(x + m * ld_x + k, (int64_t)I - (int64_t)k), hi, lo);
            const bf16x8 fw = Stage::exact8(w, c0 + weight_row<FN>(i, r), C, I, k);
            acc = mfma16(fw, lo, acc);
            acc = mfma16(fw, hi, acc);
        }
        const uint64_t c = c0 + weight_row<FN>(i, 4 * g);
        if (row < M && c < C)
            by_type(y_type, [&](auto *t) {
                store4((decltype(t))y + row * ld_y + c, acc, (int64_t)(C - c));
            });
    }
}

// y[m][c] = sum_i x[m][i] W[c][i] with W's rows staged by Stage: the
// weight's own rows for linear, its columns for the input's gradient.  fp16
// activations meet the weight in fp16; a workgroup that came upon a block
// outside fp16's range computes its tile again with exact_tiles, so that no
// weight is ever rounded.  One such block slows the whole call down to that
// tile's time: 512 x 4096 x 4096 49 -> 201 us (every tile 371), 2047 x 6400 x
// 1600 56 -> 866, the gradient 4096 x 4096 x 11008 383 -> 10,050.
template <class Fmt, template <class, uint32_t> class Stage, int FM, int FN, int AHEAD>
__global__ __launch_bounds__(kTileThreads, FM == 8 ? 2 : 4) void zs_mx_half_tile_kernel(
    const typename Fmt::T *__restrict__ x, uint64_t ld_x, MxArgs w, uint64_t M, uint64_t C,
    uint64_t I, uint32_t tm, uint32_t tc, void *y, int y_type, uint64_t ld_y, Part split) {
    constexpr uint32_t TM = 32 * FM, TC = 64 * FN;
    if (Stage<Fmt, TC>::kSplits)
        split.take(blockIdx.y, 64, x, w, M, C, I, y, y_type, ld_y);
    typedef typename Fmt::V8 V8;
    __shared__ __align__(16) uint8_t lds[2][(TM + TC) * kStepBytes];
    __shared__ uint32_t outside; // whether a block of the tile lay outside fp16
    uint32_t im, ic;
    tile_of(blockIdx.x, tm, tc, im, ic);
    const uint64_t m0 = (uint64_t)im * TM, c0 = (uint64_t)ic * TC;
    const uint32_t wave = threadIdx.x >> 6;
    const uint32_t wm = (wave & 1u) * (16 * FM), wc = (wave >> 1) * (16 * FN);
    FragAt<FN> at;
    at.init(wm, TM + wc);
    f32x4 acc[FN][FM];
#pragma unroll
    for (int i = 0; i < FN; i++)
#pragma unroll
        for (int j = 0; j < FM; j++)
            acc[i][j] = f32x4{0, 0, 0, 0};
    HalfStage<Fmt, TM> sx;
    Stage<Fmt, TC> sw;
    sx.init(x, ld_x, m0, M);
    sw.init(w, c0, C);
    if (Fmt::kType == ZERO_F16) {
        if (threadIdx.x == 0)
            outside = 0;
        __syncthreads();
    }
    // loads run AHEAD steps ahead of their use
    typename HalfStage<Fmt, TM>::Data dx[AHEAD];
    typename Stage<Fmt, TC>::Data dw[AHEAD];
    auto load = [&](auto whole, uint64_t s, uint32_t slot) {
        sx.load(whole, dx[slot], I, 64 * s);
        sw.load(whole, dw[slot], w, I, 64 * s);
    };
    auto put = [&](uint64_t s, uint32_t slot) {
        sx.store(dx[slot], lds[s & 1]);
        const bool ok = sw.store(dw[slot], lds[s & 1] + TM * kStepBytes);
        if (Fmt::kType == ZERO_F16 && !ok)
            outside = 1;
    };
    // whole: the loads' step lies inside x (else zeros past the end)
    auto step = [&](auto whole, uint64_t s, uint32_t slot) {
        run_step<FM, FN>(
            at, lds[s & 1],
            [&](auto, uint32_t i, uint32_t j, const u32x4 &fw, const u32x4 &fx) {
                acc[i][j] = mfma16(__builtin_bit_cast(V8, fw), __builtin_bit_cast(V8, fx),
                                   acc[i][j]);
            },
            [&]() { load(whole, s + AHEAD, slot); });
        put(s + 1, (slot + 1) % AHEAD); // past the last step: to where nothing is read
        __syncthreads();
    };
    const uint64_t steps = (I + 63) / 64;
#pragma unroll
    for (uint32_t d = 0; d < AHEAD; d++)
        load(Const<0>(), d, d);
    put(0, 0);
    __syncthreads();
    uint64_t s = 0;
#pragma unroll 1
    for (; 64 * (s + 2 * AHEAD) <= I; s += AHEAD)
#pragma unroll
        for (uint32_t d = 0; d < AHEAD; d++)
            step(Const<1>(), s + d, d);
#pragma unroll 1
    for (; s < steps; s += AHEAD)
#pragma unroll
        for (uint32_t d = 0; d < AHEAD; d++)
            if (d == 0 || s + d < steps)
                step(Const<0>(), s + d, d);
    if (Fmt::kType != ZERO_F16 || __builtin_amdgcn_readfirstlane(outside) == 0)
        store_tiles<FM, FN>(acc, m0 + wm, c0 + wc, M, C, y, y_type, ld_y);
    else if constexpr (Fmt::kType == ZERO_F16)
        exact_tiles<Stage<Fmt, TC>, FM, FN>(x, ld_x, w, m0 + wm, c0 + wc, M, C, I, y, y_type,
                                            ld_y);
}

// ---------------------------------------------------------------------------
// The input's gradient for up to kSkinnyM rows.  One workgroup takes 64
// columns of dx and its 16 waves (8 where more than 16 rows need the
// registers) share out the weight's rows, 32 at a time.
// Lane l reads four columns of the eight rows 8 (l / 16) + i and turns them in
// its registers: fragment e of the matrix cores' first operand is column 4
// (l % 16) + e, so that lane l of the result holds the columns 16 (l / 16) +
// 4 i + e of row l % 16 and no shared memory is needed before the join.
// ---------------------------------------------------------------------------
template <class Fmt, int MT>
struct GradSkinnyData {
    uint32_t code[8], byte[8];
    typename Fmt::V8 x[MT];
};

// The four fragments of 32 rows by 64 columns in Fmt.
template <class Fmt>
__device__ __forceinline__ void turn_columns(const uint32_t (&code)[8], const uint32_t (&byte)[8],
                                             typename Fmt::V8 (&f)[4]) {
    uint32_t v[8][2];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float s = __uint_as_float(byte[i] << 23);
        if constexpr (Fmt::kType == ZERO_F16) {
            v[i][0] = __builtin_bit_cast(uint32_t,
                                         __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i], s, 0));
            v[i][1] = __builtin_bit_cast(uint32_t,
                                         __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(code[i], s, 1));
        } else {
            v[i][0] = __builtin_bit_cast(uint32_t,
                                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], s, 0));
            v[i][1] = __builtin_bit_cast(uint32_t,
                                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code[i], s, 1));
        }
    }
#pragma unroll
    for (int e = 0; e < 4; e++) {
        const uint32_t sel = e % 2 ? 0x07060302u : 0x05040100u;
        u32x4 p;
        for (int t = 0; t < 4; t++)
            p[t] = __builtin_amdgcn_perm(v[2 * t + 1][e / 2], v[2 * t][e / 2], sel);
        f[e] = __builtin_bit_cast(typename Fmt::V8, p);
    }
}

template <class Fmt, int MT>
__global__ __launch_bounds__(grad_waves(MT) * 64) void zs_mx_grad_skinny_kernel(
    const typename Fmt::T *__restrict__ dy, uint64_t ld_dy, MxArgs w, uint64_t M, uint64_t N,
    uint64_t K, void *dx, int dx_type, uint64_t ld_dx, Part split) {
    split.take(blockIdx.y, 32, dy, w, M, K, N, dx, dx_type, ld_dx);
    constexpr uint32_t kWaves = grad_waves(MT);
    __shared__ f32x4 lds[kWaves * 4 * 64];
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x >> 6;
    const uint32_t r = lane & 15u, g = lane >> 4;
    const uint64_t k0 = (uint64_t)blockIdx.x * kGradCols, last = (K - 1) / 4u * 4u;
    const uint64_t k = k0 + 4u * r < last ? k0 + 4u * r : last;
    const uint8_t *codes = w.codes + k / 2u, *scales = w.scales + k / 32u;
    f32x4 acc[MT][4];
    for (int t = 0; t < MT; t++)
        for (int e = 0; e < 4; e++)
            acc[t][e] = f32x4{0, 0, 0, 0};
    auto load = [&](uint64_t step, GradSkinnyData<Fmt, MT> &d) {
        const uint64_t n = step * 32u + 8u * g;
        for (uint32_t i = 0; i < 8; i++) { // rows past the last one: zeros
            const uint64_t row = n + i < N ? n + i : N - 1;
            d.code[i] = *(const uint16_t *)(codes + row * w.ld_codes);
            d.byte[i] = scales[row * w.ld_scales];
        }
        for (int t = 0; t < MT; t++) {
            const uint64_t m = t * 16u + r < M ? t * 16u + r : M - 1;
            d.x[t] = load8<Fmt>(dy + m * ld_dy + n, (int64_t)N - (int64_t)n);
        }
    };
    const uint64_t steps = (N + 31) / 32;
    GradSkinnyData<Fmt, MT> d, next;
    if (wave < steps)
        load(wave, d);
    for (uint64_t step = wave; step < steps; step += kWaves) {
        if (step + kWaves < steps)
            load(step + kWaves, next);
        const uint64_t n = step * 32u + 8u * g;
        bool fits = true;
        for (uint32_t i = 0; i < 8; i++) {
            if (n + i >= N) {
                d.code[i] = 0;
                d.byte[i] = 127;
            }
            if (Fmt::kType == ZERO_F16)
                fits &= fits_f16(d.byte[i], d.code[i]);
        }
        if (Fmt::kType != ZERO_F16 || __all(fits)) {
            typename Fmt::V8 f[4];
            turn_columns<Fmt>(d.code, d.byte, f);
            for (int t = 0; t < MT; t++)
                for (int e = 0; e < 4; e++)
                    acc[t][e] = mfma16(f[e], d.x[t], acc[t][e]);
        } else if constexpr (Fmt::kType == ZERO_F16) {
            bf16x8 f[4];
            turn_columns<BF16>(d.code, d.byte, f);
            for (int t = 0; t < MT; t++) {
                bf16x8 hi, lo;
                split_f16(d.x[t], hi, lo);
                for (int e = 0; e < 4; e++) {
                    acc[t][e] = mfma16(f[e], lo, acc[t][e]);
                    acc[t][e] = mfma16(f[e], hi, acc[t][e]);
                }
            }
        }
        d = next;
    }
    // the waves' sums in order; 64 neighbours write 64 columns of a row
    const uint32_t col = lane;
    for (int t = 0; t < MT; t++) {
        for (int e = 0; e < 4; e++)
            lds[(wave * 4 + e) * 64 + lane] = acc[t][e];
        __syncthreads();
        for (uint32_t m16 = wave; m16 < 16; m16 += kWaves) {
            const float *p = (const float *)lds +
                             ((col % 4u) * 64u + col / 16u * 16u + m16) * 4u + col / 4u % 4u;
            float sum = p[0];
            for (uint32_t v = 1; v < kWaves; v++)
                sum += p[v * 1024u];
            const uint64_t m = t * 16u + m16;
            if (m < M && k0 + col < K)
                by_type(dx_type, [&](auto *o) {
                    typedef decltype(o) P;
                    ((P)dx)[m * ld_dx + k0 + col] = (typename std::remove_pointer<P>::type)sum;
                });
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// Checks and launches.
// ---------------------------------------------------------------------------
uint64_t type_bytes(int type) {
    return type == ZERO_F32 ? 4 : type == ZERO_F16 || type == ZERO_BF16 ? 2 : 0;
}

// A row-major matrix of an element type: its byte range, or an error.
int matrix_range(const void *p, int type, uint64_t rows, uint64_t cols, uint64_t ld, bool written,
                 zs::Range *r) {
    const uint64_t es = type_bytes(type);
    *r = {0, 0, written};
    if (es == 0 || ld < cols)
        return ZERO_EINVAL;
    if (rows == 0 || cols == 0)
        return ZERO_OK;
    if (!p || (uintptr_t)p % es)
        return ZERO_EINVAL;
    uint64_t b;
    if (__builtin_mul_overflow(rows - 1, ld, &b) || __builtin_add_overflow(b, cols, &b) ||
        __builtin_mul_overflow(b, es, &b) || (uintptr_t)p + b < (uintptr_t)p)
        return ZERO_EOVERFLOW;
    *r = {(uintptr_t)p, (uintptr_t)p + b, written};
    return ZERO_OK;
}

// A 4-bit matrix: the ranges of its codes and scales, or an error.
int mx_ranges(const zero_mxfp4 *q, bool written, zs::Range r[2]) {
    r[0] = r[1] = {0, 0, written};
    if (!q)
        return ZERO_EINVAL;
    const uint64_t nb = q->cols / 32 + (q->cols % 32 != 0);
    if (nb > UINT64_MAX / 32)
        return ZERO_EOVERFLOW;
    if (q->ld_codes % 16 || q->ld_codes < nb * 16 || q->ld_scales < nb)
        return ZERO_EINVAL;
    if (q->rows == 0 || q->cols == 0)
        return ZERO_OK;
    if (!q->codes || !q->scales || (uintptr_t)q->codes % 16)
        return ZERO_EINVAL;
    const uint64_t lds[2] = {q->ld_codes, q->ld_scales}, row[2] = {nb * 16, nb};
    void *const base[2] = {q->codes, q->scales};
    for (int i = 0; i < 2; i++) {
        uint64_t b;
        if (__builtin_mul_overflow(q->rows - 1, lds[i], &b) ||
            __builtin_add_overflow(b, row[i], &b) || (uintptr_t)base[i] + b < (uintptr_t)base[i])
            return ZERO_EOVERFLOW;
        r[i] = {(uintptr_t)base[i], (uintptr_t)base[i] + b, written};
    }
    return ZERO_OK;
}

int launch_status() { return hipGetLastError() == hipSuccess ? ZERO_OK : ZERO_EHIP; }

// Largest M, N and K of a product, and row pitches (in elements, or bytes
// of codes) below which an offset inside a tile fits 32 bits; offsets of
// tiles are 64-bit.
constexpr uint64_t kMaxDim = 1ull << 30;
constexpr uint64_t kMaxPitch = 1ull << 23;

MxArgs mx_args(const zero_mxfp4 *q) {
    return {(const uint8_t *)q->codes, (const uint8_t *)q->scales, q->ld_codes, q->ld_scales};
}

__global__ __launch_bounds__(256) void zs_mx_zero_kernel(uint8_t *y, uint64_t halves,
                                                         uint64_t pitch, uint64_t total) {
    const uint64_t step = (uint64_t)gridDim.x * 256u;
    for (uint64_t i = (uint64_t)blockIdx.x * 256u + threadIdx.x; i < total; i += step)
        *(uint16_t *)(y + i / halves * pitch + i % halves * 2u) = 0;
}

// y = 0 over m x n: the product over an empty K.
int zero_rows(void *y, int type, uint64_t m, uint64_t n, uint64_t ld, hipStream_t st) {
    const uint64_t es = type_bytes(type), halves = n * es / 2;
    const uint64_t total = m * halves, want = (total + 255) / 256;
    hipLaunchKernelGGL(zs_mx_zero_kernel, dim3((uint32_t)(want < 4096 ? want : 4096)), dim3(256),
                       0, st, (uint8_t *)y, halves, ld * es, total);
    return launch_status();
}

} // namespace

extern "C" int zero_mxfp4_layout(uint64_t rows, uint64_t cols, zero_mxfp4 *out) {
    if (!out)
        return ZERO_EINVAL;
    const uint64_t nb = cols / 32 + (cols % 32 != 0);
    uint64_t pitch, total;
    if (__builtin_mul_overflow(nb, (uint64_t)16, &pitch) ||
        __builtin_mul_overflow(pitch, rows, &total))
        return ZERO_EOVERFLOW;
    *out = {nullptr, nullptr, rows, cols, pitch, nb};
    return ZERO_OK;
}

extern "C" int zero_mxfp4_quantize(const void *src, int src_type, uint64_t ld_src,
                                   const zero_mxfp4 *dst, int32_t *nonfinite_flag, void *stream) {
    zs::Range r[4];
    int rc = mx_ranges(dst, true, r);
    if (rc == ZERO_OK)
        rc = matrix_range(src, src_type, dst->rows, dst->cols, ld_src, false, &r[2]);
    if (rc == ZERO_OK && (uintptr_t)nonfinite_flag % 4)
        rc = ZERO_EINVAL;
    if (rc != ZERO_OK)
        return rc;
    if (dst->rows == 0 || dst->cols == 0)
        return ZERO_OK;
    r[3] = {(uintptr_t)nonfinite_flag, (uintptr_t)nonfinite_flag + (nonfinite_flag ? 4 : 0), true};
    if (zs::writes_overlap(r, 4))
        return ZERO_EINVAL;
    uint64_t rows = dst->rows, cols = dst->cols, nb = (cols + 31) / 32;
    uint64_t blocks;
    if (__builtin_mul_overflow(rows, nb, &blocks))
        return ZERO_EOVERFLOW;
    // rows back to back in every array are one long row
    if (rows > 1 && cols % 32 == 0 && ld_src == cols && dst->ld_codes == nb * 16 &&
        dst->ld_scales == nb) {
        cols *= rows;
        nb = blocks;
        rows = 1;
    }
    const uint64_t grid = (blocks + kQuantBlocks - 1) / kQuantBlocks;
    if (grid > zs::kMaxWorkgroups256)
        return ZERO_EOVERFLOW;
    hipStream_t st = (hipStream_t)stream;
    uint8_t *c = (uint8_t *)dst->codes, *s = (uint8_t *)dst->scales;
    if (src_type == ZERO_F32)
        hipLaunchKernelGGL(zs_mx_quantize_f32_kernel, dim3((uint32_t)grid), dim3(kQuantThreads),
                           0, st, (const float *)src, ld_src, rows, cols, nb, c, dst->ld_codes, s,
                           dst->ld_scales, nonfinite_flag);
    else if (src_type == ZERO_F16)
        hipLaunchKernelGGL(zs_mx_quantize_kernel<F16>, dim3((uint32_t)grid), dim3(kQuantThreads),
                           0, st, (const _Float16 *)src, ld_src, rows, cols, nb, c, dst->ld_codes,
                           s, dst->ld_scales, nonfinite_flag);
    else
        hipLaunchKernelGGL(zs_mx_quantize_kernel<BF16>, dim3((uint32_t)grid), dim3(kQuantThreads),
                           0, st, (const __bf16 *)src, ld_src, rows, cols, nb, c, dst->ld_codes, s,
                           dst->ld_scales, nonfinite_flag);
    return launch_status();
}

static int launch_dequantize(const ShardArgs &a, uint32_t shards, uint64_t rows, uint64_t cols,
                             uint64_t ld_codes, uint64_t ld_scales, void *out, int type,
                             uint64_t ld_out, uint64_t shard_stride, hipStream_t st) {
    uint64_t nb = (cols + 31) / 32, blocks;
    if (__builtin_mul_overflow(rows, nb, &blocks))
        return ZERO_EOVERFLOW;
    if (rows > 1 && cols % 32 == 0 && ld_out == cols && ld_codes == nb * 16 && ld_scales == nb) {
        cols *= rows;
        nb = blocks;
        rows = 1;
    }
    const uint64_t grid = (blocks + kQuantBlocks - 1) / kQuantBlocks;
    if (grid > zs::kMaxWorkgroups256)
        return ZERO_EOVERFLOW;
    const dim3 g((uint32_t)grid, shards), b(kQuantThreads);
    if (type == ZERO_F32)
        hipLaunchKernelGGL(zs_mx_dequantize_kernel<F32>, g, b, 0, st, a, rows, cols, nb, ld_codes,
                           ld_scales, (float *)out, ld_out, shard_stride);
    else if (type == ZERO_F16)
        hipLaunchKernelGGL(zs_mx_dequantize_kernel<F16>, g, b, 0, st, a, rows, cols, nb, ld_codes,
                           ld_scales, (_Float16 *)out, ld_out, shard_stride);
    else
        hipLaunchKernelGGL(zs_mx_dequantize_kernel<BF16>, g, b, 0, st, a, rows, cols, nb,
                           ld_codes, ld_scales, (__bf16 *)out, ld_out, shard_stride);
    return launch_status();
}

extern "C" int zero_mxfp4_dequantize(const zero_mxfp4 *src, void *dst, int dst_type,
                                     uint64_t ld_dst, void *stream) {
    zs::Range r[3];
    int rc = mx_ranges(src, false, r);
    if (rc == ZERO_OK)
        rc = matrix_range(dst, dst_type, src->rows, src->cols, ld_dst, true, &r[2]);
    if (rc != ZERO_OK)
        return rc;
    if (src->rows == 0 || src->cols == 0)
        return ZERO_OK;
    if (zs::writes_overlap(r, 3))
        return ZERO_EINVAL;
    ShardArgs a = {};
    a.codes[0] = (const uint8_t *)src->codes;
    a.scales[0] = (const uint8_t *)src->scales;
    return launch_dequantize(a, 1, src->rows, src->cols, src->ld_codes, src->ld_scales, dst,
                             dst_type, ld_dst, 0, (hipStream_t)stream);
}

extern "C" int zero_gather_shards_mxfp4(const void *const *codes, const void *const *scales,
                                        uint32_t nd, uint64_t shard_len, void *full,
                                        int full_type, void *stream) {
    if (!codes || !scales || nd == 0 || nd > ZERO_MAX_SLICES || shard_len % 32)
        return ZERO_EINVAL;
    const uint64_t es = type_bytes(full_type);
    uint64_t n, fb;
    if (es == 0)
        return ZERO_EINVAL;
    if (__builtin_mul_overflow(shard_len, (uint64_t)nd, &n) || __builtin_mul_overflow(n, es, &fb))
        return ZERO_EOVERFLOW;
    if (shard_len == 0)
        return ZERO_OK;
    const uintptr_t f = (uintptr_t)full;
    if (!f || f % es || f + fb < f)
        return ZERO_EINVAL;
    for (uint32_t i = 0; i < nd; i++) {
        const uintptr_t c = (uintptr_t)codes[i], s = (uintptr_t)scales[i];
        const uint64_t cb = shard_len / 2, sb = shard_len / 32;
        if (!c || !s || c % 16 || c + cb < c || s + sb < s)
            return ZERO_EINVAL;
        if ((c < f + fb && f < c + cb) || (s < f + fb && f < s + sb))
            return ZERO_EINVAL;
    }
    for (uint32_t i = 0; i < nd; i += kMaxShardsPerLaunch) {
        const uint32_t count = nd - i < kMaxShardsPerLaunch ? nd - i : kMaxShardsPerLaunch;
        ShardArgs a = {};
        for (uint32_t j = 0; j < count; j++) {
            a.codes[j] = (const uint8_t *)codes[i + j];
            a.scales[j] = (const uint8_t *)scales[i + j];
        }
        const int rc = launch_dequantize(a, count, 1, shard_len, shard_len / 2, shard_len / 32,
                                         (char *)full + (uint64_t)i * shard_len * es, full_type,
                                         shard_len, shard_len, (hipStream_t)stream);
        if (rc != ZERO_OK)
            return rc;
    }
    return ZERO_OK;
}

// Sizes, ranges and overlap of a product of an m x inner matrix with w.
static int check_product(zs::Range *r, size_t n, uint64_t m, uint64_t pitch,
                         const zero_mxfp4 *w) {
    if (m > kMaxDim || w->rows > kMaxDim || w->cols > kMaxDim || pitch > kMaxPitch ||
        w->ld_codes > kMaxPitch || w->ld_scales > kMaxPitch)
        return ZERO_EOVERFLOW;
    return zs::writes_overlap(r, n) ? ZERO_EINVAL : ZERO_OK;
}

// 16-row tiles a workgroup of the skinny kernels takes: as few as hold m.
#define ZS_BY_MT(M, CALL)                                                                          \
    do {                                                                                           \
        if ((M) <= 16) {                                                                           \
            CALL(1);                                                                               \
        } else if ((M) <= 32) {                                                                    \
            CALL(2);                                                                               \
        } else {                                                                                   \
            CALL(4);                                                                               \
        }                                                                                          \
    } while (0)

static dim3 skinny_grid(uint64_t N) {
    const uint64_t groups = (N + 15) / 16;
    return groups <= kSkinnyGridX
               ? dim3((uint32_t)groups)
               : dim3((uint32_t)kSkinnyGridX, (uint32_t)((groups + kSkinnyGridX - 1) / kSkinnyGridX));
}

// Workgroups: as many as the registers let run at once, taking the groups in
// turn (dealt evenly over fewer workgroups, the CUs were not: 5 x 50257 x 1600
// 12.7 us against 11.9).
template <class Left, int OCC>
static int launch_rows(const void *x, uint64_t ld_x, MxArgs a, const zero_mxfp4 *w, uint64_t M,
                       void *y, int y_type, uint64_t ld_y, hipStream_t st) {
    const uint64_t groups = (w->rows + 15) / 16, cap = kCUs * OCC / 2;
    const uint64_t grid = groups < cap ? groups : cap;
    hipLaunchKernelGGL((zs_mx_rows_kernel<Left, OCC>), dim3((uint32_t)grid),
                       dim3(kSkinnyWaves * 64), 0, st, (const typename Left::T *)x, ld_x, a,
                       mx_args(w), M, w->rows, (uint32_t)w->cols,
                       (uint32_t)((w->cols + 31) / 32), (uint32_t)groups, y, y_type, ld_y);
    return launch_status();
}

template <int FM, int FN>
static int launch_matmul_tiles(const zero_mxfp4 *a, const zero_mxfp4 *w, void *y, int y_type,
                               uint64_t ld_y, hipStream_t st) {
    const uint64_t M = a->rows, N = w->rows;
    const uint64_t tm = (M + 32 * FM - 1) / (32 * FM), tn = (N + 64 * FN - 1) / (64 * FN);
    if (tm * tn > zs::kMaxWorkgroups512)
        return ZERO_EOVERFLOW;
    hipLaunchKernelGGL((zs_mx_matmul_tile_kernel<FM, FN>), dim3((uint32_t)(tm * tn)),
                       dim3(kTileThreads), 0, st, mx_args(a), mx_args(w), M, N,
                       (w->cols + 31) / 32, (uint32_t)tm, (uint32_t)tn, y, y_type, ld_y);
    return launch_status();
}

extern "C" int zero_mxfp4_matmul(const zero_mxfp4 *a, const zero_mxfp4 *w, void *y, int y_type,
                                 uint64_t ld_y, void *stream) {
    zs::Range r[5];
    int rc = mx_ranges(a, false, r);
    if (rc == ZERO_OK)
        rc = mx_ranges(w, false, r + 2);
    if (rc != ZERO_OK)
        return rc;
    if (a->cols != w->cols)
        return ZERO_EINVAL;
    const uint64_t M = a->rows, N = w->rows, K = w->cols, nb = (K + 31) / 32;
    if ((rc = matrix_range(y, y_type, M, N, ld_y, true, &r[4])) != ZERO_OK ||
        (rc = check_product(r, 5, M, a->ld_codes > a->ld_scales ? a->ld_codes : a->ld_scales, w)) !=
            ZERO_OK)
        return rc;
    if (M == 0 || N == 0)
        return ZERO_OK;
    hipStream_t st = (hipStream_t)stream;
    if (K == 0)
        return zero_rows(y, y_type, M, N, ld_y, st);
    if (!skinny(M, N)) {
        switch (tile_frags(M, N, kLeastTilesMx)) {
        case 8:
            return launch_matmul_tiles<8, 4>(a, w, y, y_type, ld_y, st);
        case 4:
            return launch_matmul_tiles<4, 2>(a, w, y, y_type, ld_y, st);
        default:
            return launch_matmul_tiles<2, 1>(a, w, y, y_type, ld_y, st);
        }
    }
#define ZS_CALL(S, MT, OCC)                                                                        \
    return launch_rows<LeftMx<S, MT>, OCC>(nullptr, 0, mx_args(a), w, M, y, y_type, ld_y, st)
    if (M <= 16 && in_registers(nb, 2))
        ZS_CALL(2, 1, 8);
    if (M <= 16 && in_registers(nb, 4))
        ZS_CALL(4, 1, 6);
    if (M <= 16 && in_registers(nb, 8))
        ZS_CALL(8, 1, 4);
    if (M <= 16 && in_registers(nb, 12))
        ZS_CALL(12, 1, 2);
    if (M <= 32 && in_registers(nb, 2))
        ZS_CALL(2, 2, 8);
    if (M <= 32 && in_registers(nb, 4))
        ZS_CALL(4, 2, 4);
#undef ZS_CALL
    const dim3 grid = skinny_grid(N);
#define ZS_CALL(MT)                                                                                \
    hipLaunchKernelGGL((zs_mx_matmul_skinny_kernel<MT>), grid, dim3(kSkinnyWaves * 64), 0, st,     \
                       mx_args(a), mx_args(w), M, N, (uint32_t)nb, y, y_type, ld_y)
    ZS_BY_MT(M, ZS_CALL);
#undef ZS_CALL
    return launch_status();
}

template <class Fmt, template <class, uint32_t> class Stage, int FM, int FN, int AHEAD>
static int launch_half_tiles(const void *x, uint64_t ld_x, const zero_mxfp4 *w, uint64_t M,
                             uint64_t C, uint64_t I, void *y, int y_type, uint64_t ld_y,
                             const Part &split, hipStream_t st) {
    const uint64_t tm = (M + 32 * FM - 1) / (32 * FM), tc = (C + 64 * FN - 1) / (64 * FN);
    if (tm * tc > zs::kMaxWorkgroups512)
        return ZERO_EOVERFLOW;
    hipLaunchKernelGGL((zs_mx_half_tile_kernel<Fmt, Stage, FM, FN, AHEAD>),
                       dim3((uint32_t)(tm * tc), split.parts), dim3(kTileThreads), 0, st,
                       (const typename Fmt::T *)x, ld_x, mx_args(w), M, C, I, (uint32_t)tm,
                       (uint32_t)tc, y, y_type, ld_y, split);
    return launch_status();
}

template <class Fmt, template <class, uint32_t> class Stage>
static int half_tiles(const void *x, uint64_t ld_x, const zero_mxfp4 *w, uint64_t M, uint64_t C,
                      uint64_t I, void *y, int y_type, uint64_t ld_y, const Part &split,
                      hipStream_t st) {
    switch (tile_frags(M, C, kLeastTilesHalf)) {
    case 8:
        return launch_half_tiles<Fmt, Stage, 8, 4, 1>(x, ld_x, w, M, C, I, y, y_type, ld_y, split,
                                                       st);
    case 4:
        return launch_half_tiles<Fmt, Stage, 4, 2, 1>(x, ld_x, w, M, C, I, y, y_type, ld_y, split,
                                                       st);
    default:
        return launch_half_tiles<Fmt, Stage, 2, 1, 4>(x, ld_x, w, M, C, I, y, y_type, ld_y, split,
                                                       st);
    }
}

template <class Fmt>
static int linear(const void *x, uint64_t m, uint64_t ld_x, const zero_mxfp4 *w, void *y,
                  int y_type, uint64_t ld_y, hipStream_t st) {
    const uint64_t N = w->rows, K = w->cols, nb = (K + 31) / 32;
    if (!skinny(m, N))
        return half_tiles<Fmt, RowStage>(x, ld_x, w, m, N, K, y, y_type, ld_y, {1, nullptr}, st);
#define ZS_CALL(S, MT, OCC)                                                                        \
    return launch_rows<LeftRows<Fmt, S, MT>, OCC>(x, ld_x, MxArgs{}, w, m, y, y_type, ld_y, st)
    if (m <= 16 && in_registers(nb, 2))
        ZS_CALL(2, 1, 6);
    if (m <= 16 && in_registers(nb, 4))
        ZS_CALL(4, 1, 4);
    if (m <= 16 && in_registers(nb, 8))
        ZS_CALL(8, 1, 2);
    if (m <= 32 && in_registers(nb, 2))
        ZS_CALL(2, 2, 4);
    if (m <= 32 && in_registers(nb, 4))
        ZS_CALL(4, 2, 2);
#undef ZS_CALL
    const dim3 grid = skinny_grid(N);
#define ZS_CALL(MT)                                                                                \
    hipLaunchKernelGGL((zs_mx_linear_skinny_kernel<Fmt, MT>), grid, dim3(kSkinnyWaves * 64), 0,    \
                       st, (const typename Fmt::T *)x, ld_x, mx_args(w), m, N, (uint32_t)K,        \
                       (uint32_t)nb, y, y_type, ld_y)
    ZS_BY_MT(m, ZS_CALL);
#undef ZS_CALL
    return launch_status();
}

extern "C" int zero_mxfp4_linear(const void *x, int x_type, uint64_t m, uint64_t ld_x,
                                 const zero_mxfp4 *w, void *y, int y_type, uint64_t ld_y,
                                 void *stream) {
    zs::Range r[4];
    int rc = mx_ranges(w, false, r);
    if (rc != ZERO_OK)
        return rc;
    if (x_type != ZERO_F16 && x_type != ZERO_BF16)
        return ZERO_EINVAL;
    if ((rc = matrix_range(x, x_type, m, w->cols, ld_x, false, &r[2])) != ZERO_OK ||
        (rc = matrix_range(y, y_type, m, w->rows, ld_y, true, &r[3])) != ZERO_OK ||
        (rc = check_product(r, 4, m, ld_x, w)) != ZERO_OK)
        return rc;
    if (m == 0 || w->rows == 0)
        return ZERO_OK;
    hipStream_t st = (hipStream_t)stream;
    if (w->cols == 0)
        return zero_rows(y, y_type, m, w->rows, ld_y, st);
    return x_type == ZERO_F16 ? linear<F16>(x, m, ld_x, w, y, y_type, ld_y, st)
                              : linear<BF16>(x, m, ld_x, w, y, y_type, ld_y, st);
}

template <class Fmt>
static int grad_input(const void *dy, uint64_t m, uint64_t ld_dy, const zero_mxfp4 *w, void *dx,
                      int dx_type, uint64_t ld_dx, const Part &split, hipStream_t st) {
    const uint64_t N = w->rows, K = w->cols;
    int rc;
    if (m > kSkinnyM) {
        rc = half_tiles<Fmt, ColumnStage>(dy, ld_dy, w, m, K, N, dx, dx_type, ld_dx, split, st);
    } else {
        const uint64_t grid = (K + kGradCols - 1) / kGradCols;
        if (grid > zs::kMaxWorkgroups1024)
            return ZERO_EOVERFLOW;
#define ZS_CALL(MT)                                                                                \
    hipLaunchKernelGGL((zs_mx_grad_skinny_kernel<Fmt, MT>), dim3((uint32_t)grid, split.parts),     \
                       dim3(grad_waves(MT) * 64), 0, st, (const typename Fmt::T *)dy, ld_dy,       \
                       mx_args(w), m, N, K, dx, dx_type, ld_dx, split)
        ZS_BY_MT(m, ZS_CALL);
#undef ZS_CALL
        rc = launch_status();
    }
    if (rc != ZERO_OK || split.parts == 1)
        return rc;
    const dim3 g((uint32_t)((K + 255) / 256), (uint32_t)m), b(256);
    if (dx_type == ZERO_F32)
        hipLaunchKernelGGL(zs_mx_join_kernel<float>, g, b, 0, st, split.partial, split.parts, m, K,
                           (float *)dx, ld_dx);
    else if (dx_type == ZERO_F16)
        hipLaunchKernelGGL(zs_mx_join_kernel<_Float16>, g, b, 0, st, split.partial, split.parts, m,
                           K, (_Float16 *)dx, ld_dx);
    else
        hipLaunchKernelGGL(zs_mx_join_kernel<__bf16>, g, b, 0, st, split.partial, split.parts, m,
                           K, (__bf16 *)dx, ld_dx);
    return launch_status();
}

extern "C" int zero_mxfp4_grad_workspace(uint64_t m, const zero_mxfp4 *w, uint64_t *bytes) {
    if (!w || !bytes)
        return ZERO_EINVAL;
    if (m > kMaxDim || w->rows > kMaxDim || w->cols > kMaxDim)
        return ZERO_EOVERFLOW;
    const uint32_t parts = m && w->rows && w->cols ? grad_parts(m, w->rows, w->cols) : 1;
    *bytes = parts > 1 ? parts * m * w->cols * 4 : 0;
    return ZERO_OK;
}

extern "C" int zero_mxfp4_linear_grad_input(const void *dy, int dy_type, uint64_t m,
                                            uint64_t ld_dy, const zero_mxfp4 *w, void *dx,
                                            int dx_type, uint64_t ld_dx, void *workspace,
                                            uint64_t workspace_bytes, void *stream) {
    zs::Range r[5];
    int rc = mx_ranges(w, false, r);
    if (rc != ZERO_OK)
        return rc;
    if ((dy_type != ZERO_F16 && dy_type != ZERO_BF16) || (uintptr_t)workspace % 4 ||
        (!workspace && workspace_bytes))
        return ZERO_EINVAL;
    if ((uintptr_t)workspace + workspace_bytes < (uintptr_t)workspace)
        return ZERO_EOVERFLOW;
    r[4] = {0, 0, true}; // no bytes overlap nothing
    if (workspace_bytes)
        r[4] = {(uintptr_t)workspace, (uintptr_t)workspace + workspace_bytes, true};
    if ((rc = matrix_range(dy, dy_type, m, w->rows, ld_dy, false, &r[2])) != ZERO_OK ||
        (rc = matrix_range(dx, dx_type, m, w->cols, ld_dx, true, &r[3])) != ZERO_OK ||
        (rc = check_product(r, 5, m, ld_dy, w)) != ZERO_OK)
        return rc;
    if (m == 0 || w->cols == 0)
        return ZERO_OK;
    hipStream_t st = (hipStream_t)stream;
    if (w->rows == 0)
        return zero_rows(dx, dx_type, m, w->cols, ld_dx, st);
    // as many parts as the workspace holds
    const uint64_t fit = workspace_bytes / (m * w->cols * 4);
    const uint32_t parts = grad_parts(m, w->rows, w->cols);
    const Part split = {fit < 2 ? 1 : fit < parts ? (uint32_t)fit : parts, (float *)workspace};
    return dy_type == ZERO_F16
               ? grad_input<F16>(dy, m, ld_dy, w, dx, dx_type, ld_dx, split, st)
               : grad_input<BF16>(dy, m, ld_dy, w, dx, dx_type, ld_dx, split, st);
}
