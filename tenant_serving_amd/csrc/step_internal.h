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

// kv.hip
struct Strides2 {
    int64_t token, head;
};
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
};
hipError_t launch_attend(const AttendArgs& a, bool q_fp32, hipStream_t stream);

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
