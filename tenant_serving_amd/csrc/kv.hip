// The paged key-value cache's rows, written (rounded to bf16, or held as e4m3
// codes with one power-of-two scale) and read back.
//
// Bound by HBM: every row is read once and written once.  A row is held by a
// group of neighbouring lanes, 8 values each (the group rounded up to a power
// of two), so a row's largest magnitude takes log2(lanes) exchanges and no
// shared memory.
#include "step_internal.h"

namespace bd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 64;  // of one workgroup of the write

struct WriteArgs {
    bd_kv kv;
    const void* k;
    const void* v;
    Strides2 ks, vs;
    const int32_t* slots;
    int32_t T;
    int32_t per;  // tokens of a workgroup
    int32_t capacity;
};

// A workgroup writes the rows of `per` neighbouring tokens.  Where a later
// token names the same slot, that one's rows are to stay, whatever order the
// workgroups run in: so a workgroup first looks for its own slots among the
// later ones.  It reads them once, and compares only those inside the range
// its own slots span (a page or two in a prefill), which keeps the search at
// a few percent of the copy.
template <bool kX32, bool kE4m3, int kLanes>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(const WriteArgs a) {
    __shared__ int own[kMaxTokens];
    __shared__ int dead[kMaxTokens];
    __shared__ int range[2];
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * a.per;
    const int n = a.T - t0 < a.per ? (int)(a.T - t0) : a.per;

    if (tid < 64) {
        int s = tid < n ? a.slots[t0 + tid] : -1;
        if (s >= a.capacity) s = -1;
        own[tid] = s;
        dead[tid] = s < 0;
        // -1 counts as the largest number below, as no number above
        unsigned lo = (unsigned)s;
        int hi = s;
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const unsigned l = (unsigned)__shfl_xor((int)lo, off, 64);
            const int h = __shfl_xor(hi, off, 64);
            lo = l < lo ? l : lo;
            hi = h > hi ? h : hi;
        }
        if (tid == 0) range[0] = (int)(lo > 0x7fffffffu ? 0x7fffffffu : lo), range[1] = hi;
    }
    __syncthreads();
    const int lo = range[0], hi = range[1];
    for (int64_t t = t0 + 1 + tid; t < a.T; t += kThreads) {
        const int s = a.slots[t];
        if (s < lo || s > hi) continue;
        const int before = t - t0 < n ? (int)(t - t0) : n;
        for (int i = 0; i < before; ++i)
            if (own[i] == s) dead[i] = 1;  // every writer writes 1
    }
    __syncthreads();

    const int lane = tid % kLanes;
    const int e = lane * 8;
    const bool in = e < a.kv.head_dim;
    const int H = a.kv.num_heads;
    const int rows = n * 2 * H;
    for (int r = tid / kLanes; r < rows; r += kThreads / kLanes) {
        const int i = r / (2 * H);
        const int hv = r - i * 2 * H;
        const bool is_v = hv >= H;
        const int head = is_v ? hv - H : hv;
        Raw8<kX32> raw;
        raw.zero();
        const Strides2 st = is_v ? a.vs : a.ks;
        if (in) raw.load(is_v ? a.v : a.k, (t0 + i) * st.token + head * st.head + e);
        float f[8];
        raw.widen(f);
        if (dead[i]) continue;  // whole row groups of lanes
        const int slot = own[i];
        const int page = slot / a.kv.page_size, at = slot - page * a.kv.page_size;
        const int64_t to = page * a.kv.page_stride + head * a.kv.head_stride + at * a.kv.token_stride + e;
        if (kE4m3) {
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t b = finite_bits(f[j]);
                top = b > top ? b : top;
            }
#pragma unroll
            for (int off = 1; off < kLanes; off <<= 1) {
                const uint32_t o = (uint32_t)__shfl_xor((int)top, off, 64);
                top = o > top ? o : top;
            }
            const int byte = scale_byte(top);
            const float inv = inv_scale_of(byte);
            if (in) {
                const uint2 w = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3], inv),
                                           pack_e4m3x4(f[4], f[5], f[6], f[7], inv));
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.kv.v : a.kv.k) + to) = w;
            }
            if (lane == 0)
                (is_v ? a.kv.v_scales : a.kv.k_scales)[((int64_t)page * H + head) * a.kv.page_size + at] =
                    (uint8_t)byte;
        } else if (in) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.kv.v : a.kv.k) + to) = narrow_bf16x8(f);
        }
    }
}

struct ReadArgs {
    bd_kv kv;
    const int32_t* slots;
    uint16_t* k_out;
    uint16_t* v_out;
    int64_t rows;  // T * num_heads
    int32_t capacity;
};

// One row group per (token, head), keys in grid row 0 and values in 1.
template <bool kE4m3, int kLanes>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(const ReadArgs a) {
    const int tid = threadIdx.x;
    const int64_t r = (int64_t)blockIdx.x * (kThreads / kLanes) + tid / kLanes;
    const int e = (tid % kLanes) * 8;
    if (r >= a.rows || e >= a.kv.head_dim) return;
    const bool is_v = blockIdx.y != 0;
    const int64_t t = r / a.kv.num_heads;
    const int head = (int)(r - t * a.kv.num_heads);
    const int slot = a.slots[t];
    uint4 w = make_uint4(0, 0, 0, 0);
    if (slot >= a.capacity) {
        w = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    } else if (slot >= 0) {
        const int page = slot / a.kv.page_size, at = slot - page * a.kv.page_size;
        const int64_t from = page * a.kv.page_stride + head * a.kv.head_stride + at * a.kv.token_stride + e;
        if (kE4m3) {
            const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(is_v ? a.kv.v : a.kv.k) + from);
            const float s = scale_of(
                (is_v ? a.kv.v_scales : a.kv.k_scales)[((int64_t)page * a.kv.num_heads + head) * a.kv.page_size + at]);
            w = make_uint4(e4m3x2_to_bf16<false>(c.x, s), e4m3x2_to_bf16<true>(c.x, s), e4m3x2_to_bf16<false>(c.y, s),
                           e4m3x2_to_bf16<true>(c.y, s));
        } else {
            w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(is_v ? a.kv.v : a.kv.k) + from);
        }
    }
    *reinterpret_cast<uint4*>((is_v ? a.v_out : a.k_out) + r * a.kv.head_dim + e) = w;
}

template <bool kX32, bool kE4m3>
void write_lanes(const WriteArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + a.per - 1) / a.per)), block(kThreads);
    const int lanes = a.kv.head_dim / 8;
    if (lanes <= 8)
        hipLaunchKernelGGL((kv_write_kernel<kX32, kE4m3, 8>), grid, block, 0, s, a);
    else if (lanes <= 16)
        hipLaunchKernelGGL((kv_write_kernel<kX32, kE4m3, 16>), grid, block, 0, s, a);
    else
        hipLaunchKernelGGL((kv_write_kernel<kX32, kE4m3, 32>), grid, block, 0, s, a);
}

template <bool kE4m3>
void read_lanes(ReadArgs a, hipStream_t s) {
    const int lanes = a.kv.head_dim / 8 <= 8 ? 8 : a.kv.head_dim / 8 <= 16 ? 16 : 32;
    const int64_t per = kThreads / lanes;
    const int64_t all = a.rows / a.kv.num_heads;                                    // tokens
    const int64_t most = (int64_t(1) << 23) * per / a.kv.num_heads;                 // of one launch: threads below 2^32
    for (int64_t t0 = 0; t0 < all; t0 += most) {
        ReadArgs b = a;
        const int64_t n = all - t0 < most ? all - t0 : most;
        b.slots += t0;
        b.k_out += t0 * a.kv.num_heads * a.kv.head_dim;
        b.v_out += t0 * a.kv.num_heads * a.kv.head_dim;
        b.rows = n * a.kv.num_heads;
        const dim3 grid((unsigned)((b.rows + per - 1) / per), 2), block(kThreads);
        if (lanes == 8)
            hipLaunchKernelGGL((kv_read_kernel<kE4m3, 8>), grid, block, 0, s, b);
        else if (lanes == 16)
            hipLaunchKernelGGL((kv_read_kernel<kE4m3, 16>), grid, block, 0, s, b);
        else
            hipLaunchKernelGGL((kv_read_kernel<kE4m3, 32>), grid, block, 0, s, b);
    }
}

}  // namespace

hipError_t launch_kv_write(const bd_kv& kv, const void* k, Strides2 ks, const void* v, Strides2 vs, bool fp32,
                           const int32_t* slots, int64_t T, hipStream_t stream) {
    const int64_t per = (T + 2047) / 2048;
    const WriteArgs a{kv, k, v, ks, vs, slots, (int32_t)T, (int32_t)(per < kMaxTokens ? per : kMaxTokens),
                      (int32_t)(kv.num_pages * kv.page_size)};
    if (kv.type == BD_E4M3) {
        if (fp32)
            write_lanes<true, true>(a, stream);
        else
            write_lanes<false, true>(a, stream);
    } else {
        if (fp32)
            write_lanes<true, false>(a, stream);
        else
            write_lanes<false, false>(a, stream);
    }
    return hipGetLastError();
}

hipError_t launch_kv_read(const bd_kv& kv, const int32_t* slots, int64_t T, uint16_t* k_out, uint16_t* v_out,
                          hipStream_t stream) {
    const ReadArgs a{kv, slots, k_out, v_out, T * kv.num_heads, (int32_t)(kv.num_pages * kv.page_size)};
    if (kv.type == BD_E4M3)
        read_lanes<true>(a, stream);
    else
        read_lanes<false>(a, stream);
    return hipGetLastError();
}

}  // namespace bd
