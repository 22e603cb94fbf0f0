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

// What is read back is stored streaming where it is more than the 256 MiB
// last-level cache would keep for the next kernel: 65536 tokens (268 MB) 80.7 ->
// 73.5 us, with a kernel that reads it after 153.9 -> 145.5; at 32768 plain stores
// win with that kernel (65.4 against 70.5; right behind the write of the same
// tokens the two are within 3% from 4096 to 32768).  What is written to the cache, never:
// a prefill reads it right after (16384 tokens from fp32 to e4m3 37.0 -> 35.1 us,
// but their read-back 16.6 -> 20.9).
constexpr int64_t kStreamBytes = int64_t(192) << 20;
template <bool kStream>
__device__ __forceinline__ void store16(uint16_t* p, uint4 v) {
    const u32x4_t w = {v.x, v.y, v.z, v.w};
    if (kStream)
        __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
    else
        *reinterpret_cast<u32x4_t*>(p) = w;
}

constexpr int kThreads = 256;   // of the read
// Rows that a lane of the read holds at once, of keys and of values each.
// 131071 tokens of 8 heads of 128 in e4m3, against one row of either array per
// lane and plain stores: 192 -> 142 us (5.7 TB/s); one row 147, four 145.
constexpr int kReadRows = 2;
// The write: up to kSmallWrite tokens by workgroups of 256 lanes (1..2 tokens
// each), more by at most 1024 of 1024 lanes (up to 32 tokens each), in slices.
// Fewer and larger workgroups read the later slots fewer times, but start on
// the rows later: 16384 tokens from fp32 to e4m3 with 512 / 1024 / 2048 of them
// 39.3 / 38.2 / 47.3 us; 65536 in slices of 16384 / 32768 / 65536 157 / 162 / 155,
// from bf16 125 / 118 / 126, and a slice bounds what the search costs a token.
constexpr int64_t kSmallWrite = 4096;
constexpr int64_t kSmallGroups = 2048, kGroups = 1024;
constexpr int64_t kSlice = 32768;
static_assert(kSmallWrite <= 2 * kSmallGroups && kSlice <= 32 * kGroups, "tables of kv_write_kernel");

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

struct WriteArgs {
    bd_kv kv;
    const void* k;
    const void* v;
    Strides2 ks, vs;
    const int32_t* slots;
    Div page, row;  // by page_size, by the rows of a token (keys, then values)
    int32_t T;
    int32_t per;  // tokens of a workgroup
    int32_t capacity;
};

// The largest of kLanes neighbouring lanes' numbers, in all of them.
template <int kCtrl>
__device__ __forceinline__ uint32_t max_dpp(uint32_t x) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)x, (int)x, kCtrl, 0xf, 0xf, false);
    return o > x ? o : x;
}
template <int kLanes>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
    x = max_dpp<0xb1>(x);                       // quads: lane ^ 1
    x = max_dpp<0x4e>(x);                       // lane ^ 2
    x = max_dpp<0x141>(x);                      // mirrored within 8: the other quad
    if (kLanes >= 16) x = max_dpp<0x140>(x);    // mirrored within 16: the other half
    if (kLanes == 32) {
        const uint32_t o = (uint32_t)__shfl_xor((int)x, 16, 64);
        x = o > x ? o : x;
    }
    return x;
}

// A workgroup writes the rows of `per` neighbouring tokens.  Where a later
// token names the same slot, that one's rows are to stay, whatever order the
// workgroups run in: so a workgroup first looks for its own slots among the
// later ones (2 us of 38 at 16384 tokens), while its first rows are on their
// way.  A slot outside the range of its own (256 lanes, where these are one or
// two), or without their bit in a table of 65536 (1024 lanes), is none of
// them; the rest are compared.
template <bool kX32, bool kE4m3, int kLanes, int kWide>
__global__ __launch_bounds__(kWide) void kv_write_kernel(const WriteArgs a) {
    constexpr int kMost = kWide == 256 ? 2 : 32;  // tokens of a workgroup
    __shared__ int own[kMost], dead[kMost];
    __shared__ int64_t to_row[kMost], to_scale[kMost];
    __shared__ int range[2];
    constexpr int kBits = 65536;
    __shared__ uint32_t bits[kWide == 256 ? 1 : kBits / 32];
    const auto hash = [](int s) { return (uint32_t)s * 0x9e3779b1u >> 16; };
    constexpr int kPer = kWide / kLanes;  // rows at a time
    const int tid = threadIdx.x;
    const int64_t t0 = (int64_t)blockIdx.x * a.per;
    const int n = a.T - t0 < a.per ? (int)(a.T - t0) : a.per;
    const int lane = tid % kLanes, e = lane * 8, r0 = tid / kLanes;
    const bool in = e < a.kv.head_dim;
    const int H = a.kv.num_heads;
    const int rows = n * 2 * H;

    Raw8<kX32> raw;
    const auto load = [&](int r) {
        raw.zero();
        if (in && r < rows) {
            const int i = (int)a.row.by((uint32_t)r), hv = r - i * 2 * H;
            const bool is_v = hv >= H;
            const Strides2 st = is_v ? a.vs : a.ks;
            raw.load(is_v ? a.v : a.k, (t0 + i) * st.token + (is_v ? hv - H : hv) * st.head + e);
        }
    };
    load(r0);

    if (kWide == 256) {
        if (tid == 0) range[0] = -1, range[1] = -1;
    } else {
        for (int i = tid; i < kBits / 32; i += kWide) bits[i] = 0;
    }
    __syncthreads();
    if (tid < kMost) {
        int s = tid < n ? a.slots[t0 + tid] : -1;
        if (s >= a.capacity || s < 0) s = -1;
        own[tid] = s;
        dead[tid] = s < 0;
        const int page = s < 0 ? 0 : (int)a.page.by((uint32_t)s), at = s < 0 ? 0 : s - page * a.kv.page_size;
        to_row[tid] = page * a.kv.page_stride + at * a.kv.token_stride;
        to_scale[tid] = (int64_t)page * H * a.kv.page_size + at;
        if (s >= 0) {
            if (kWide == 256) {  // as unsigned, -1 is above every slot
                atomicMin(reinterpret_cast<unsigned*>(&range[0]), (unsigned)s);
                atomicMax(&range[1], s);
            } else {
                const uint32_t h = hash(s);
                atomicOr(&bits[h >> 5], 1u << (h & 31));
            }
        }
    }
    __syncthreads();
    {
        const int lo = kWide == 256 ? range[0] : 0;
        const uint32_t width = kWide == 256 ? (uint32_t)range[1] - (uint32_t)lo : 0u;
        const auto maybe = [&](int s) -> bool {
            if (kWide == 256) return lo >= 0 && (uint32_t)s - (uint32_t)lo <= width;
            const uint32_t h = hash(s);
            return (bits[h >> 5] >> (h & 31)) & 1;
        };
        // among its own: every pair, kMost a power of two
        for (int p = tid; p < n * kMost; p += kWide) {
            const int i = p & (kMost - 1), j = p / kMost;
            if (i < j && own[i] == own[j]) dead[i] = 1;  // every writer writes 1
        }
        // among the later ones
        const auto look = [&](int s) {
            for (int i = 0; i < n; ++i)
                if (own[i] == s && s >= 0) dead[i] = 1;
        };
        // up to a 16-byte border, whole 16 bytes, the rest
        const int64_t start = t0 + n;
        const int64_t odd = (int64_t)((reinterpret_cast<uintptr_t>(a.slots + start) >> 2) & 3);
        int64_t body = start + ((4 - odd) & 3);
        if (body > a.T) body = a.T;
        const int vecs = (int)((a.T - body) >> 2);
        const int64_t rest = body + (int64_t)vecs * 4;
        if (start + tid < body) look(a.slots[start + tid]);
        if (rest + tid < a.T) look(a.slots[rest + tid]);
        const int4* body4 = reinterpret_cast<const int4*>(a.slots + body);
#pragma unroll 2
        for (int v = tid; v < vecs; v += kWide) {
            const int4 s = body4[v];
            const bool x = maybe(s.x), y = maybe(s.y), z = maybe(s.z), w = maybe(s.w);
            if (x || y || z || w) {
#pragma nounroll
                for (int i = 0; i < 4; ++i)
                    if (i == 0 ? x : i == 1 ? y : i == 2 ? z : w)
                        look(i == 0 ? s.x : i == 1 ? s.y : i == 2 ? s.z : s.w);
            }
        }
    }
    __syncthreads();

    for (int r = r0; r < rows; r += kPer) {  // whole groups of lanes
        float f[8];
        raw.widen(f);
        load(r + kPer);
        const int i = (int)a.row.by((uint32_t)r), hv = r - i * 2 * H;
        const bool is_v = hv >= H;
        const int head = is_v ? hv - H : hv;
        const int64_t to = to_row[i] + head * a.kv.head_stride + e;
        const bool keep = !dead[i];
        if (kE4m3) {
            uint32_t top = 0;
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const uint32_t b = finite_bits(f[x]);
                top = b > top ? b : top;
            }
            top = group_max<kLanes>(top);
            const int byte = scale_byte(top);
            const float inv = inv_scale_of(byte);
            if (in && keep) {
                const uint2 w = make_uint2(pack_e4m3x4(f[0], f[1], f[2], f[3], inv),
                                           pack_e4m3x4(f[4], f[5], f[6], f[7], inv));
                *reinterpret_cast<uint2*>(static_cast<uint8_t*>(is_v ? a.kv.v : a.kv.k) + to) = w;
            }
            if (lane == 0 && keep)
                (is_v ? a.kv.v_scales : a.kv.k_scales)[to_scale[i] + (int64_t)head * a.kv.page_size] = (uint8_t)byte;
        } else if (in && keep) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.kv.v : a.kv.k) + to) = narrow_bf16x8(f);
        }
    }
}

// Eight held values: bf16, or codes and their row's scale byte.
template <bool kE4m3>
struct Held;
template <>
struct Held<false> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const void* p, int64_t i, const uint8_t*, int64_t) {
        w = load_stream16(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    }
    __device__ __forceinline__ uint4 value() const { return w; }
};
template <>
struct Held<true> {
    uint2 w;
    int byte;
    __device__ __forceinline__ void zero() { w = make_uint2(0, 0), byte = 127; }
    __device__ __forceinline__ void load(const void* p, int64_t i, const uint8_t* scales, int64_t s) {
        w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + i);
        byte = scales[s];
    }
    __device__ __forceinline__ uint4 value() const {
        const float s = scale_of(byte);
        return make_uint4(e4m3x2_to_bf16<false>(w.x, s), e4m3x2_to_bf16<true>(w.x, s), e4m3x2_to_bf16<false>(w.y, s),
                          e4m3x2_to_bf16<true>(w.y, s));
    }
};

struct ReadArgs {
    bd_kv kv;
    const int32_t* slots;
    uint16_t* k_out;
    uint16_t* v_out;
    int64_t rows;  // T * num_heads, below 2^31
    Div page, head;
    int32_t capacity;
};

// A lane reads its piece of kRows rows of keys and of as many rows of values
// before it writes any of them.
template <bool kE4m3, int kLanes, bool kStream>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(const ReadArgs a) {
    constexpr int kPer = kThreads / kLanes;  // rows at a time
    const int e = ((int)threadIdx.x % kLanes) * 8;
    if (e >= a.kv.head_dim) return;
    const int64_t r0 = (int64_t)blockIdx.x * (kPer * kReadRows) + threadIdx.x / kLanes;
    Held<kE4m3> x[kReadRows][2];
    int slot[kReadRows];
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int64_t r = r0 + i * kPer;
        x[i][0].zero();
        x[i][1].zero();
        slot[i] = -1;
        if (r < a.rows) {
            const uint32_t t = a.head.by((uint32_t)r), head = (uint32_t)r - t * a.kv.num_heads;
            slot[i] = a.slots[t];
            if (slot[i] >= 0 && slot[i] < a.capacity) {
                const int page = (int)a.page.by((uint32_t)slot[i]), at = slot[i] - page * a.kv.page_size;
                const int64_t from = page * a.kv.page_stride + head * a.kv.head_stride + at * a.kv.token_stride + e;
                const int64_t sc = ((int64_t)page * a.kv.num_heads + head) * a.kv.page_size + at;
                x[i][0].load(a.kv.k, from, a.kv.k_scales, sc);
                x[i][1].load(a.kv.v, from, a.kv.v_scales, sc);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kReadRows; ++i) {
        const int64_t r = r0 + i * kPer;
        if (r >= a.rows) break;
        const bool past = slot[i] >= a.capacity;
        const uint4 nan = make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
        store16<kStream>(a.k_out + r * a.kv.head_dim + e, past ? nan : x[i][0].value());
        store16<kStream>(a.v_out + r * a.kv.head_dim + e, past ? nan : x[i][1].value());
    }
}

template <bool kX32, bool kE4m3, int kLanes>
void write_wide(const WriteArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.T + a.per - 1) / a.per));
    if (a.T <= kSmallWrite)
        hipLaunchKernelGGL((kv_write_kernel<kX32, kE4m3, kLanes, 256>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((kv_write_kernel<kX32, kE4m3, kLanes, 1024>), grid, dim3(1024), 0, s, a);
}

template <bool kX32, bool kE4m3>
void write_lanes(const WriteArgs& a, hipStream_t s) {
    const int lanes = a.kv.head_dim / 8;
    if (lanes <= 8)
        write_wide<kX32, kE4m3, 8>(a, s);
    else if (lanes <= 16)
        write_wide<kX32, kE4m3, 16>(a, s);
    else
        write_wide<kX32, kE4m3, 32>(a, s);
}

template <bool kE4m3, bool kStream>
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
        const dim3 grid((unsigned)((b.rows + per * kReadRows - 1) / (per * kReadRows))), block(kThreads);
        if (lanes == 8)
            hipLaunchKernelGGL((kv_read_kernel<kE4m3, 8, kStream>), grid, block, 0, s, b);
        else if (lanes == 16)
            hipLaunchKernelGGL((kv_read_kernel<kE4m3, 16, kStream>), grid, block, 0, s, b);
        else
            hipLaunchKernelGGL((kv_read_kernel<kE4m3, 32, kStream>), grid, block, 0, s, b);
    }
}

template <bool kE4m3>
void read_any(const ReadArgs& a, hipStream_t s) {
    if (a.rows * a.kv.head_dim * 4 >= kStreamBytes)
        read_lanes<kE4m3, true>(a, s);
    else
        read_lanes<kE4m3, false>(a, s);
}

}  // namespace

hipError_t launch_kv_write(const bd_kv& kv, const void* k, Strides2 ks, const void* v, Strides2 vs, bool fp32,
                           const int32_t* slots, int64_t T, hipStream_t stream) {
    // Long calls in slices, one after another on the stream: a later slice's
    // rows come over an earlier one's by themselves, and a workgroup's search
    // stays within its slice.
    for (int64_t t0 = 0; t0 < T; t0 += kSlice) {
        const int64_t n = T - t0 < kSlice ? T - t0 : kSlice;
        const bool small = n <= kSmallWrite;
        int64_t per = small ? (n + kSmallGroups - 1) / kSmallGroups : (n + kGroups - 1) / kGroups;
        // 64 rows at least, which 1024 lanes take at once at head_dim 128: few
        // heads would leave the search to more workgroups than their rows are
        // worth
        const int64_t least = small ? 1 : 32 / kv.num_heads;
        if (per < least) per = least;
        const int64_t size = fp32 ? 4 : 2;
        const WriteArgs a{kv, static_cast<const char*>(k) + t0 * ks.token * size,
                          static_cast<const char*>(v) + t0 * vs.token * size, ks, vs, slots + t0,
                          Div((uint32_t)kv.page_size), Div((uint32_t)(2 * kv.num_heads)), (int32_t)n, (int32_t)per,
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
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_kv_read(const bd_kv& kv, const int32_t* slots, int64_t T, uint16_t* k_out, uint16_t* v_out,
                          hipStream_t stream) {
    const ReadArgs a{kv, slots, k_out, v_out, T * kv.num_heads, Div((uint32_t)kv.page_size),
                     Div((uint32_t)kv.num_heads), (int32_t)(kv.num_pages * kv.page_size)};
    if (kv.type == BD_E4M3)
        read_any<true>(a, stream);
    else
        read_any<false>(a, stream);
    return hipGetLastError();
}

}  // namespace bd
