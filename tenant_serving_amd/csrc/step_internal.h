// Host-side launch entry points of the operators between the linears of a
// step (include/bitdelta_step.h), and the device code their kernels share.
// The ABI layer (step_api.cpp) validates every argument before calling these.
#pragma once

#include "bd_device.h"
#include "../../include/bitdelta_step.h"

namespace bd {

// api.cpp: the current device is a gfx950 GPU (else its bd_status), and its
// number of compute units.
bd_status check_current_device(int* num_cu);

// norm.hip
constexpr int64_t kNormMaxD = 65536;
struct NormArgs {
    const void* x;
    const void* residual;
    void* residual_out;
    const void* gain;
    const int32_t* ids;  // may be null
    void* out;
    uint8_t* scales;
    float eps;
    int32_t num_gains;
    int32_t gain_fp32;
    int32_t d;
    int64_t M;
};
// x_fp32; residual: 0 none, 1 bf16, 2 fp32
hipError_t launch_norm(const NormArgs& a, bool x_fp32, int residual, bool e4m3, hipStream_t stream);

struct Strides2 {
    int64_t token, head;
};

// n / d for 0 <= n < 2^31 by a product: m = ceil(2^s / d) with s = 31 + ceil(log2 d)
// is below 2^32 and too large by less than d / 2^s, which n cannot carry over.
struct Div {
    uint32_t d, m, shift;  // shift: s - 32
    __host__ explicit Div(uint32_t by) : d(by) {
        int up = 0;
        while ((uint64_t(1) << up) < by) ++up;
        m = (uint32_t)(((uint64_t(1) << (31 + up)) + by - 1) / by);
        shift = up > 0 ? up - 1 : 0;
        if (up == 0) m = 0;  // by 1: see by()
    }
    __device__ __forceinline__ uint32_t by(uint32_t n) const { return m ? __umulhi(n, m) >> shift : n; }
};

// rotary.hip
struct RotaryArgs {
    const void* x[2];
    void* out[2];
    Strides2 xs[2], os[2];
    int32_t heads[2];  // the second 0 where there is one tensor
    const int32_t* positions;
    const uint64_t* steps;
    float gain;
    int32_t dim, turned;
    int64_t T;
};
hipError_t launch_rotary(const RotaryArgs& a, bool x_fp32, bool out_fp32, bool interleaved, hipStream_t stream);

// kv.hip
hipError_t launch_kv_write(const bd_kv& kv, const void* k, Strides2 ks, const void* v, Strides2 vs, bool fp32,
                           const int32_t* slots, int64_t T, hipStream_t stream);
hipError_t launch_kv_read(const bd_kv& kv, const int32_t* slots, int64_t T, uint16_t* k_out, uint16_t* v_out,
                          hipStream_t stream);

// attend.hip
constexpr int64_t kAttendMaxTokens = int64_t(1) << 24;  // per sequence
size_t attend_workspace_bytes(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages);
struct AttendArgs {
    bd_kv kv;
    const void* q;
    Strides2 qs;
    const int32_t* table;
    const int32_t* lengths;
    uint16_t* out;
    float* lse;   // may be null
    float* part;  // workspace, may be null where nothing is split
    int64_t table_stride;
    int32_t max_pages, B, Hq;
    float scale;
    float cap;             // 0: none
    const float* slopes;   // may be null
    const int32_t* first;  // may be null
};
hipError_t launch_attend(const AttendArgs& a, bool q_fp32, hipStream_t stream);

// prompt.hip
size_t prompt_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t capacity);
struct PromptArgs {
    bd_kv kv;
    const uint16_t* q;
    Strides2 qs;
    const int32_t* table;
    const int32_t* lengths;
    const int32_t* starts;
    uint16_t* out;
    float* lse;   // may be null
    float* part;  // workspace, may be null where nothing is split
    int64_t table_stride;
    int32_t max_pages, B, T, Hq;
    float scale;
    float cap;             // 0: none
    const float* slopes;   // may be null
    const int32_t* first;  // may be null
    const int32_t* last;   // may be null
};
hipError_t launch_prompt(const PromptArgs& a, hipStream_t stream);

// Capped scores in units of their cap: x = tanh(times x), times = scale / cap.
// tanh y = 1 - 2 / (1 + e^(2 y)) loses what is small against 1, and costs two
// quarter-rate operations.  Where |y| <= 1/2 it is y + y^3 g(y^2), g of degree 3
// fitted to the least relative error of the whole (2^-25.7); that is the usual
// case, as scores are small against a cap, and the only one where all of a
// wave's scores are.  Where some are larger each lane takes what suits it.
// A shorter g would give lse, an fp32 result, an error that grows with the cap:
// degree 2 (2^-20.5) that of 12 roundings of the score.
template <int kN>
__device__ __forceinline__ void cap_scores(float* x, float times) {
    float big = 0.0f;
    float small[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
        const float y = x[j] = x[j] * times;
        big = fmaxf(big, __builtin_fabsf(y));
        const float q = y * y;
        float g = __builtin_fmaf(q, 0.017257417f, -0.05305313f);
        g = __builtin_fmaf(g, q, 0.13325989f);
        g = __builtin_fmaf(g, q, -0.3333315f);
        small[j] = __builtin_fmaf(g, q * y, y);
    }
    if (__ballot(!(big <= 0.5f))) {
#pragma unroll
        for (int j = 0; j < kN; ++j) {
            const float e = __builtin_amdgcn_exp2f(x[j] * 2.8853900817779268f);  // 2 log2(e)
            const float t = __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + e), 1.0f);
            x[j] = __builtin_fabsf(x[j]) <= 0.5f ? small[j] : t;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kN; ++j) x[j] = small[j];
    }
}
// What formed scores are kept in: units of the cap, or of 1 without one.  `times`
// makes them of products (of the queries with scale's sign).
struct Form {
    float unit, times;
};
inline Form form_of(float scale, float cap) {
    const float size = scale < 0.0f ? -scale : scale, unit = cap > 0.0f ? cap : 1.0f;
    // an infinite product times a scale other than 0 stays infinite
    return Form{unit, size > 0.0f && size / unit == 0.0f ? 0x1p-149f : size / unit};
}
// A slope in these units; finite, so that it takes nothing off at no distance.
__device__ __forceinline__ float slope_in(float slope, float unit) {
    return __builtin_amdgcn_fmed3f(slope / unit, -0x1.fffffep127f, 0x1.fffffep127f);
}

// ---------------------------------------------------------------------------
// e4m3 groups

constexpr int kMinScaleByte = 16;  // 2^-111: every code times its scale is a normal bf16 number

// The bits of |x| where x is finite, else 0: what a group's largest magnitude
// is taken over.  Their order as whole numbers is the magnitudes' order.
__device__ __forceinline__ uint32_t finite_bits(float x) {
    const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
    return b < 0x7f800000u ? b : 0u;
}
// The scale byte of a group whose largest magnitude has these bits: the
// exponent field, one more where the mantissa exceeds 448's (1.75 * 2^8;
// adding 0x1fffff carries into the exponent exactly then), less 8.
__device__ __forceinline__ int scale_byte(uint32_t bits) {
    const int b = (int)((bits + 0x1fffffu) >> 23) - 8;
    return b < kMinScaleByte ? kMinScaleByte : b;
}
// 2^(byte - 127) and its inverse; the byte is 16 .. 247 there, so both are normal.
__device__ __forceinline__ float scale_of(int byte) { return __uint_as_float((uint32_t)byte << 23); }
__device__ __forceinline__ float inv_scale_of(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Four values times inv -> four e4m3 codes (v_cvt_pk_fp8_f32, nearest even).
// Infinities become NaN here (infinity times zero), since the conversion's own
// answer for them depends on a mode bit.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d, float inv) {
    const auto prep = [&](float x) {
        const float t = x * inv;
        return __builtin_fmaf(t, 0.0f, t);
    };
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(prep(a), prep(b), 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(prep(c), prep(d), r, true);
    return (uint32_t)r;
}

// Two e4m3 codes (the low or high half of a dword) times a power of two ->
// packed bf16 pair, exactly (v_cvt_scalef32_pk_bf16_fp8).
template <bool kHigh>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, kHigh));
}

// ---------------------------------------------------------------------------
// e2m1 groups

constexpr int kGroup4 = 32;        // values of a group
constexpr int kMinScaleByte4 = 2;  // 2^-125: half of it, the least code but 0, is a normal bf16 number
constexpr int kNanByte = 255;

// The scale byte of a group whose largest magnitude has these bits (6 = 1.5 * 2^2).
__device__ __forceinline__ int scale_byte4(uint32_t bits) {
    if (bits >= 0x7f800000u) return kNanByte;
    const int b = (int)((bits + 0x3fffffu) >> 23) - 2;
    return b < kMinScaleByte4 ? kMinScaleByte4 : b;
}
// Eight values times inv (the inverse of their scale, by which they are exact
// but below the least code) -> eight e2m1 codes (v_cvt_scalef32_pk_fp4_f32,
// nearest even).
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* f, float inv) {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0] * inv, f[1] * inv, 1.0f, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2] * inv, f[3] * inv, 1.0f, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4] * inv, f[5] * inv, 1.0f, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6] * inv, f[7] * inv, 1.0f, 3);
    return r;
}
// Two e2m1 codes (byte kByte of a dword) times the power of two whose exponent
// scale has -> packed bf16 pair, exactly (v_cvt_scalef32_pk_bf16_fp4; an
// exponent of 255 gives NaN, one of 0 is 2^-127).
template <int kByte>
__device__ __forceinline__ uint32_t e2m1x2_to_bf16(uint32_t codes, float scale) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, kByte));
}
__device__ __forceinline__ uint4 e2m1x8_to_bf16(uint32_t codes, float scale) {
    return make_uint4(e2m1x2_to_bf16<0>(codes, scale), e2m1x2_to_bf16<1>(codes, scale),
                      e2m1x2_to_bf16<2>(codes, scale), e2m1x2_to_bf16<3>(codes, scale));
}

// ---------------------------------------------------------------------------
// Eight consecutive values as fp32.
__device__ __forceinline__ void widen_bf16x8(uint4 w, float* f) {
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        f[2 * p] = __uint_as_float(ws[p] << 16);
        f[2 * p + 1] = __uint_as_float(ws[p] & 0xffff0000u);
    }
}
// Raw registers of eight values: one 16-byte load of bf16, two of fp32.
template <bool kFp32>
struct Raw8;
template <>
struct Raw8<false> {
    uint4 a;
    __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    }
    __device__ __forceinline__ void load_stream(const void* p, int64_t i) {
        a = load_stream16(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
    __device__ __forceinline__ void widen(float* f) const { widen_bf16x8(a, f); }
};
template <>
struct Raw8<true> {
    float4 a, b;
    __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        a = q[0];
        b = q[1];
    }
    __device__ __forceinline__ void load_stream(const void* p, int64_t i) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        a = load_stream16(q);
        b = load_stream16(q + 1);
    }
    __device__ __forceinline__ void widen(float* f) const {
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
        f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
};
__device__ __forceinline__ uint4 narrow_bf16x8(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

}  // namespace bd
