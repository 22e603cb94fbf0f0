// Rotary positions: the first columns of each query and key row turned in pairs.
//
//   a' = g (a cos t - b sin t),  b' = g (b cos t + a sin t),  t = 2 pi p s_i / 2^64
//
// Bound by HBM: every row is read once and written once, queries and keys in
// one launch.  A pair's angle is the same for all heads of a token, so a lane
// works it out once and goes over several rows of its token with it.
//
// The angle in whole numbers: s_i is the part of a turn that one position adds
// as a fraction of 2^64, and the low 64 bits of p s_i are the angle without its
// whole turns, however far p is.  Their upper 32 bits less the nearest quarter
// turn leave at most pi / 4, where the series of sine and cosine end soon; in fp32
// that is off by three roundings, 1.4e-7, which the results' own are as large as.
#include "step_internal.h"

namespace bd {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;  // rows that a lane holds at once

struct Args {
    RotaryArgs a;
    Div lanes, sets;       // by the lanes of a row, by the sets of rows of a token
    int32_t rows;          // of a token: both tensors' heads
    int64_t items;         // lanes in all
};

// sine and cosine of pos * step of a turn: after the nearest quarter turn is
// taken off, the Taylor series up to x^9 and x^10, whose next terms are below
// 2^-28 of the result for |x| <= pi / 4.
__device__ __forceinline__ void sine_cosine(int pos, uint2 step, float& s, float& c) {
    uint32_t turn = (uint32_t)pos * step.y + __umulhi((uint32_t)pos, step.x);
    if (pos < 0) turn -= step.x;
    const uint32_t quarter = (turn + 0x20000000u) >> 30;
    const float x = (float)(int)(turn - (quarter << 30)) * 1.4629180792671596e-09f;  // 2 pi / 2^32
    const float y = x * x;
    float a = __builtin_fmaf(y, 2.7557319e-06f, -1.9841270e-04f);
    a = __builtin_fmaf(a, y, 8.3333333e-03f);
    a = __builtin_fmaf(a, y, -1.6666667e-01f);
    const float sn = __builtin_fmaf(a * y, x, x);
    float b = __builtin_fmaf(y, -2.7557319e-07f, 2.4801587e-05f);
    b = __builtin_fmaf(b, y, -1.3888889e-03f);
    b = __builtin_fmaf(b, y, 4.1666667e-02f);
    b = __builtin_fmaf(b, y, -0.5f);
    const float cs = __builtin_fmaf(b, y, 1.0f);
    s = quarter & 1 ? cs : sn;
    c = quarter & 1 ? sn : cs;
    if (quarter & 2) s = -s;
    if ((quarter + 1) & 2) c = -c;
}

// kN consecutive values as fp32, in memory bf16 or fp32.
template <bool kFp32, int kN>
struct Values {
    static constexpr int kWords = kFp32 ? kN : (kN + 1) / 2;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const void* p, int64_t i) {
        const char* at = static_cast<const char*>(p) + i * (kFp32 ? 4 : 2);
        if constexpr (kN * (kFp32 ? 4 : 2) == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(at);
        } else if constexpr (kWords >= 4) {
#pragma unroll
            for (int v = 0; v < kWords / 4; ++v) {
                const uint4 x = reinterpret_cast<const uint4*>(at)[v];
                w[4 * v] = x.x, w[4 * v + 1] = x.y, w[4 * v + 2] = x.z, w[4 * v + 3] = x.w;
            }
        } else if constexpr (kWords == 2) {
            const uint2 x = *reinterpret_cast<const uint2*>(at);
            w[0] = x.x, w[1] = x.y;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(at);
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if (kFp32) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void set(const float* f) {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = kFp32 ? __float_as_uint(f[i]) : pack_bf16x2(f[2 * i], 2 * i + 1 < kN ? f[2 * i + 1] : 0.0f);
    }
    __device__ __forceinline__ void store(void* p, int64_t i) const {
        char* at = static_cast<char*>(p) + i * (kFp32 ? 4 : 2);
        if constexpr (kN * (kFp32 ? 4 : 2) == 2) {
            *reinterpret_cast<uint16_t*>(at) = (uint16_t)w[0];
        } else if constexpr (kWords >= 4) {
#pragma unroll
            for (int v = 0; v < kWords / 4; ++v)
                reinterpret_cast<uint4*>(at)[v] = make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
        } else if constexpr (kWords == 2) {
            *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
        } else {
            *reinterpret_cast<uint32_t*>(at) = w[0];
        }
    }
};

// A lane takes kN pairs, or 2 kN columns that stay: dim / (2 kN) lanes to a
// row.  kN: the largest power of two up to 8 that divides turned / 2, so that
// no lane's columns end inside the turned ones.
template <bool kX32, bool kO32, bool kInter, int kN>
__global__ __launch_bounds__(kThreads) void rotary_kernel(const Args p) {
    const int64_t item = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (item >= p.items) return;
    const uint32_t set_of = p.lanes.by((uint32_t)item);
    const int lane = (int)((uint32_t)item - set_of * p.lanes.d);
    const int t = (int)p.sets.by(set_of), set = (int)(set_of - (uint32_t)t * p.sets.d);
    const int half = p.a.turned / 2;
    const bool turns = lane * kN < half;
    // the lane's two pieces of kN columns
    int c0, c1;
    if (kInter || !turns) {
        c0 = lane * 2 * kN;
        c1 = c0 + kN;
    } else {
        c0 = lane * kN;
        c1 = half + c0;
    }
    float sn[kN], cs[kN];
    if (turns) {
        const int pos = p.a.positions[t];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            sine_cosine(pos, reinterpret_cast<const uint2*>(p.a.steps)[lane * kN + i], sn[i], cs[i]);
            sn[i] *= p.a.gain;
            cs[i] *= p.a.gain;
        }
    }
    const int step = (int)p.sets.d;
    for (int r0 = set; r0 < p.rows; r0 += step * kRows) {
        Values<kX32, kN> x[kRows][2];
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * step;
            if (r < p.rows) {
                const int w = r >= p.a.heads[0], h = w ? r - p.a.heads[0] : r;
                const int64_t at = t * p.a.xs[w].token + h * p.a.xs[w].head;
                x[i][0].load(p.a.x[w], at + c0);
                x[i][1].load(p.a.x[w], at + c1);
            }
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int r = r0 + i * step;
            if (r >= p.rows) break;
            const int w = r >= p.a.heads[0], h = w ? r - p.a.heads[0] : r;
            const int64_t at = t * p.a.os[w].token + h * p.a.os[w].head;
            float f[2 * kN];
#pragma unroll
            for (int j = 0; j < kN; ++j) f[j] = x[i][0].get(j), f[kN + j] = x[i][1].get(j);
            if (turns) {
#pragma unroll
                for (int j = 0; j < kN; ++j) {
                    // interleaved pairs lie side by side, others kN apart
                    float& a = f[kInter ? 2 * j : j];
                    float& b = f[kInter ? 2 * j + 1 : kN + j];
                    const float a0 = a;
                    a = __builtin_fmaf(a0, cs[j], -(b * sn[j]));
                    b = __builtin_fmaf(b, cs[j], a0 * sn[j]);
                }
            }
            Values<kO32, kN> y;
            y.set(f);
            y.store(p.a.out[w], at + c0);
            y.set(f + kN);
            y.store(p.a.out[w], at + c1);
        }
    }
}

template <bool kX32, bool kO32, bool kInter>
hipError_t go(RotaryArgs a, hipStream_t s) {
    const int half = a.turned / 2;
    const int n = half % 8 == 0 ? 8 : half % 4 == 0 ? 4 : half % 2 == 0 ? 2 : 1;
    const int rows = a.heads[0] + a.heads[1], lanes = a.dim / (2 * n);
    // rows of a lane: enough lanes to fill the GPU first, then as many rows as
    // share an angle, kRows at a time
    const int64_t wide = (int64_t)256 * 2048;
    int64_t per = a.T * rows * lanes / wide;
    per = per < 1 ? 1 : per > 2 * kRows ? 2 * kRows : per;
    const int sets = (int)((rows + per - 1) / per);
    // tokens of a launch: items below 2^31
    int64_t most = ((int64_t(1) << 31) - kThreads) / ((int64_t)sets * lanes);
    for (int64_t t0 = 0; t0 < a.T; t0 += most) {
        const int64_t n_t = a.T - t0 < most ? a.T - t0 : most;
        Args p{a, Div((uint32_t)lanes), Div((uint32_t)sets), rows, n_t * sets * lanes};
        for (int i = 0; i < 2; ++i) {
            if (a.heads[i] == 0) continue;
            p.a.x[i] = static_cast<const char*>(a.x[i]) + t0 * a.xs[i].token * (kX32 ? 4 : 2);
            p.a.out[i] = static_cast<char*>(a.out[i]) + t0 * a.os[i].token * (kO32 ? 4 : 2);
        }
        p.a.positions = a.positions + t0;
        const dim3 grid((unsigned)((p.items + kThreads - 1) / kThreads)), block(kThreads);
        switch (n) {
            case 8: hipLaunchKernelGGL((rotary_kernel<kX32, kO32, kInter, 8>), grid, block, 0, s, p); break;
            case 4: hipLaunchKernelGGL((rotary_kernel<kX32, kO32, kInter, 4>), grid, block, 0, s, p); break;
            case 2: hipLaunchKernelGGL((rotary_kernel<kX32, kO32, kInter, 2>), grid, block, 0, s, p); break;
            default: hipLaunchKernelGGL((rotary_kernel<kX32, kO32, kInter, 1>), grid, block, 0, s, p);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool kX32, bool kO32>
hipError_t go_layout(const RotaryArgs& a, bool interleaved, hipStream_t s) {
    return interleaved ? go<kX32, kO32, true>(a, s) : go<kX32, kO32, false>(a, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs& a, bool x_fp32, bool out_fp32, bool interleaved, hipStream_t stream) {
    if (x_fp32) return out_fp32 ? go_layout<true, true>(a, interleaved, stream) : go_layout<true, false>(a, interleaved, stream);
    return out_fp32 ? go_layout<false, true>(a, interleaved, stream) : go_layout<false, false>(a, interleaved, stream);
}

}  // namespace bd
