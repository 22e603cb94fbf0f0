// RMS norm with the residual's addition in front, a bf16 or an e4m3 result.
//
//   h = x + residual, kept as residual_out; y = h / sqrt(mean(h^2) + eps) * g
//
// Bound by HBM: a row is read once, stays in the registers of the lanes that
// read it (8 consecutive values per lane and chunk) while its sum of squares
// is taken, and is written once.  The mean is over the values that the
// residual stream holds afterwards, so a rounding to bf16 comes before it.
// Sums are fp32: each lane's own values in order, then a butterfly over the
// wave, then the waves' sums in wave order.
//
// A group of 32 columns of the e4m3 result is four neighbouring lanes, whose
// largest magnitude two lane exchanges give.  For this result the sums and
// products are 64-bit: in 32 bits a few codes in a million fall on the other
// side of their border.  The extra work hides behind the memory where there is a
// residual (8192 x 8192 with an fp32 one 134.9 us in 32 bits, 134.5 in 64);
// without one it is what bounds the call (2048 x 16384 from bf16 33 us, 3.1 TB/s).
#include "step_internal.h"

#include <type_traits>

namespace bd {
namespace {

// A double cut to fp32, the last bit set where that dropped anything: what is
// rounded to fewer bits from there (and a comparison with numbers of fewer bits)
// comes out as from the double.
__device__ __forceinline__ float to_odd(double y) {
    const float f = (float)y;
    const double back = (double)f;
    const uint32_t cut = __float_as_uint(f) - (uint32_t)(fabs(back) > fabs(y));
    return __uint_as_float(cut | (uint32_t)(back != y));
}

template <int NT>
constexpr int kNormBlock = NT == 64 ? 256 : NT;

// x and a bf16 residual are loaded streaming from this many bytes of them on,
// as little of them can still be in the 256 MiB last-level cache then: 2048 x
// 28672 of bf16 94 -> 82 us (5.7 TB/s), 8192 x 8192 with fp32 x 118 -> 106; below,
// what the linear just wrote is found there (2048 x 8192 with fp32 x, 100 MB,
// 29.6 against 30.8 us).  Narrow rows gain 0 to 6% (1048576 x 128 of bf16 324 ->
// 304, 262144 x 512 with fp32 x 234 -> 224, 65536 x 2048 232 -> 227; to e4m3
// they are level).  With an fp32 residual plain loads stay ahead (8192 x 8192 to
// e4m3 135 against 141), without one they are level.
constexpr int64_t kStreamBytes = int64_t(192) << 20;

// kRes: 0 no residual, 1 bf16, 2 fp32.  NT lanes own a row (64: four rows to a
// workgroup, one per wave), C chunks of 8 values each.
template <bool kX32, int kRes, bool kE4m3, bool kStream, int NT, int C>
__global__ __launch_bounds__(kNormBlock<NT>) void norm_kernel(const NormArgs a, int64_t row0) {
    const int tid = NT == 64 ? (int)threadIdx.x & 63 : (int)threadIdx.x;
    const int64_t row = row0 + (NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x);
    if (NT == 64 && row >= a.M) return;  // a whole wave; this form has no barrier
    const int64_t base = row * a.d;
    typedef typename std::conditional<kE4m3, double, float>::type Sum;

    Raw8<kX32> xr[C];
    Raw8<kRes == 2> rr[C];
    Raw8<false> gb[C];
    const int id = a.ids ? a.ids[row] : 0;
    const bool known = id >= 0 && id < a.num_gains;
    const int64_t gbase = known ? (int64_t)id * a.d : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (c * NT + tid) * 8;
        xr[c].zero();
        rr[c].zero();
        if (e < a.d) {
            if (kStream)
                xr[c].load_stream(a.x, base + e), rr[c].load_stream(a.residual, base + e);
            else
                xr[c].load(a.x, base + e);
            if (kRes && !kStream) rr[c].load(a.residual, base + e);
        }
    }
    if (!a.gain_fp32) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (c * NT + tid) * 8;
            gb[c].zero();
            if (e < a.d) gb[c].load(a.gain, gbase + e);
        }
    }

    float h[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (c * NT + tid) * 8;
        xr[c].widen(h[c]);
        if (kRes) {
            float r[8];
            rr[c].widen(r);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[c][i] += r[i];
            if (kRes == 1) {
                const uint4 w = narrow_bf16x8(h[c]);
                if (e < a.d) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.residual_out) + base + e) = w;
                widen_bf16x8(w, h[c]);
            } else if (e < a.d) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.residual_out) + base + e);
                p[0] = make_float4(h[c][0], h[c][1], h[c][2], h[c][3]);
                p[1] = make_float4(h[c][4], h[c][5], h[c][6], h[c][7]);
            }
        }
    }
    // the mean square of the row times `by`, in all of its lanes
    __shared__ Sum part[2][NT / 64];
    const auto mean_square = [&](int turn, Sum by) {
        Sum sum = 0;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const Sum x = (Sum)h[c][i] * by;
                sum = fma(x, x, sum);
            }
        }
        sum = wave_sum(sum);
        if (NT > 64) {
            if ((tid & 63) == 0) part[turn][tid >> 6] = sum;
            __syncthreads();
            sum = 0;
            if constexpr (kE4m3) {
#pragma unroll
                for (int w = 0; w < NT / 64; ++w) sum += part[turn][w];
            } else {  // through one register, not one for each wave
                const int of = __float_as_int(part[turn][tid & (NT / 64 - 1)]);
#pragma unroll
                for (int w = 0; w < NT / 64; ++w) sum += __int_as_float(__builtin_amdgcn_readlane(of, w));
            }
        }
        return sum / (Sum)a.d;
    };
    Sum under = mean_square(0, 1) + (Sum)a.eps;
    // Squares past fp32's range, or so small that they lose bits or vanish and
    // eps does not cover it: the row times a power of two, and eps times its
    // square, give the same y.  2^-76 takes the sum of 65536 of the largest
    // squares to 2^120; 2^90 takes one below 65536 times 2^-80 to 2^116, and the
    // least square to 2^-118.  Every lane of the row has the same sum and takes
    // the same way.
    float by = 1.0f;
    if constexpr (!kE4m3) {
        const float all = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(under)));
        if (all > 0x1p100f || all < 0x1p-80f) {
            by = all > 1.0f ? 0x1p-76f : 0x1p90f;
            under = mean_square(1, by) + a.eps * by * by;
        }
    }
    const Sum rstd = known ? (Sum)1 / sqrt(under) : (Sum)__builtin_nanf("");

#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (c * NT + tid) * 8;
        float g[8];
        if (a.gain_fp32) {
            Raw8<true> gw;
            gw.zero();
            if (e < a.d) gw.load(a.gain, gbase + e);
            gw.widen(g);
        } else {
            gb[c].widen(g);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (kE4m3)
                h[c][i] = to_odd((double)h[c][i] * rstd * (double)g[i]);
            else
                h[c][i] = h[c][i] * by * rstd * g[i];
        }
        if (kE4m3) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = __float_as_uint(h[c][i]) & 0x7fffffffu;
                top = b > top ? b : top;
            }
            if (__ballot(top >= 0x7f800000u)) {  // rare: what is not finite does not count
                top = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t b = finite_bits(h[c][i]);
                    top = b > top ? b : top;
                }
            }
            // lanes past d hold zeros (or NaN, which counts as 0)
#pragma unroll
            for (int off = 1; off <= 2; off <<= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)top, off, 64);
                top = o > top ? o : top;
            }
            const int byte = known ? scale_byte(top) : 127;
            const float inv = inv_scale_of(byte);
            if (e < a.d) {
                const uint2 w = make_uint2(pack_e4m3x4(h[c][0], h[c][1], h[c][2], h[c][3], inv),
                                           pack_e4m3x4(h[c][4], h[c][5], h[c][6], h[c][7], inv));
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.out) + base + e) = w;
                if ((tid & 3) == 0) a.scales[row * ((a.d + 31) / 32) + e / 32] = (uint8_t)byte;
            }
        } else if (e < a.d) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + base + e) = narrow_bf16x8(h[c]);
        }
    }
}

template <bool kX32, int kRes, bool kE4m3, bool kStream, int NT, int C>
void go(const NormArgs& a, hipStream_t s) {
    constexpr int64_t most = int64_t(1) << 21;  // rows of one launch: its threads number below 2^32
    for (int64_t row0 = 0; row0 < a.M; row0 += most) {
        const int64_t n = a.M - row0 < most ? a.M - row0 : most;
        const unsigned grid = (unsigned)(NT == 64 ? (n + 3) / 4 : n);
        hipLaunchKernelGGL((norm_kernel<kX32, kRes, kE4m3, kStream, NT, C>), dim3(grid), dim3(kNormBlock<NT>), 0, s, a,
                           row0);
    }
}

// Few lanes with several chunks each: their loads are in flight together, and a
// CU holds several rows.  2048 rows in e4m3 with an fp32 residual, this choice
// against twice the lanes or the next power of two of chunks: 6000 wide 30.5 ->
// 28.3 us, 9272 53.8 -> 43.4, 12000 66.2 -> 52.1, 16384 81.5 -> 78.2; past 16384
// 512 lanes would lose (28672 156.5 -> 165.5).  Past 32768 columns 8 chunks are
// more than the 128 registers of 1024 lanes hold in most forms: 1024 x 65536 runs
// at 2.9 to 5.8 TB/s to bf16 and 1.3 to 2.3 to e4m3.
template <bool kX32, int kRes, bool kE4m3, bool kStream>
void pick(const NormArgs& a, hipStream_t s) {
    if (a.d <= 512) return go<kX32, kRes, kE4m3, kStream, 64, 1>(a, s);
    if (a.d <= 2048) return go<kX32, kRes, kE4m3, kStream, 256, 1>(a, s);
    if (a.d <= 4096) return go<kX32, kRes, kE4m3, kStream, 256, 2>(a, s);
    if (a.d <= 6144) return go<kX32, kRes, kE4m3, kStream, 256, 3>(a, s);
    if (a.d <= 8192) return go<kX32, kRes, kE4m3, kStream, 256, 4>(a, s);
    if (a.d <= 12288) return go<kX32, kRes, kE4m3, kStream, 512, 3>(a, s);
    if (a.d <= 16384) return go<kX32, kRes, kE4m3, kStream, 512, 4>(a, s);
    if (a.d <= 24576) return go<kX32, kRes, kE4m3, kStream, 1024, 3>(a, s);
    if (a.d <= 32768) return go<kX32, kRes, kE4m3, kStream, 1024, 4>(a, s);
    return go<kX32, kRes, kE4m3, kStream, 1024, 8>(a, s);
}

template <bool kX32, int kRes>
void pick_out(const NormArgs& a, bool e4m3, hipStream_t s) {
    if constexpr (kRes == 1) {
        if (a.M * a.d * (kX32 ? 6 : 4) >= kStreamBytes) {
            if (e4m3)
                return pick<kX32, kRes, true, true>(a, s);
            return pick<kX32, kRes, false, true>(a, s);
        }
    }
    if (e4m3)
        pick<kX32, kRes, true, false>(a, s);
    else
        pick<kX32, kRes, false, false>(a, s);
}

template <bool kX32>
void pick_res(const NormArgs& a, int residual, bool e4m3, hipStream_t s) {
    if (residual == 0)
        pick_out<kX32, 0>(a, e4m3, s);
    else if (residual == 1)
        pick_out<kX32, 1>(a, e4m3, s);
    else
        pick_out<kX32, 2>(a, e4m3, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool x_fp32, int residual, bool e4m3, hipStream_t stream) {
    if (x_fp32)
        pick_res<true>(a, residual, e4m3, stream);
    else
        pick_res<false>(a, residual, e4m3, stream);
    return hipGetLastError();
}

}  // namespace bd
