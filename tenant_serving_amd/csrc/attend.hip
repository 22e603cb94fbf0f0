// Attention of one new token per sequence: the shape of a launch, its dispatch,
// and the join of rows that several workgroups worked on.  The kernel and what
// bounds it: attend_device.h.
#include "attend_device.h"

#include <algorithm>

namespace bd {
using namespace attend;
namespace {

// Adds a partial result (maximum m, sum l, unnormalised output x) to a running
// one.  A part whose scores are all -infinity has sum and output 0 (or NaN).
__device__ __forceinline__ void add_part(float c, float& M, float& L, float4& o, float m, float l, float4 x) {
    const float to = fmaxf(M, m);
    const float f = M == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((M - to) * c);
    const float g = m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((m - to) * c);
    M = to;
    L = L * f + l * g;
    o.x = o.x * f + x.x * g, o.y = o.y * f + x.y * g, o.z = o.z * f + x.z * g, o.w = o.w * f + x.w * g;
}

// Rows of units that several workgroups worked on: out = sum of their partial
// outputs over the sum of their sums, each scaled to the common maximum.  A
// row's outputs are shared out over grid y, 4 values of one head to an item; the
// lanes that a workgroup has beyond its items share out the partial results.
// Bound by latency: the table's entry, then the partial results (1 row of 57908
// tokens, 5 heads of 128, e4m3, 453 of them: a workgroup per head 11.6 us, one
// per 8 items, whose lanes' sums are added in pairs, 6.0).
__global__ __launch_bounds__(256) void join_kernel(const Args p) {
    __shared__ float4 red[256];
    __shared__ float redm[256], redl[256];
    const Cross cross = reinterpret_cast<const Cross*>(p.a.part)[blockIdx.x];
    if (cross.first < 0) return;
    const int w0 = cross.first >> 1, w1 = cross.last, which0 = cross.first & 1;
    const int b = cross.id / p.s.rows, row = cross.id - b * p.s.rows;
    const int head = row / p.s.tiles, q0 = (row - head * p.s.tiles) * 16;
    const int nq = p.s.group - q0 < 16 ? p.s.group - q0 : 16;
    const int lanes = p.s.dim / 4, all = nq * lanes;
    const int first = all * (int)blockIdx.y / (int)gridDim.y;
    const int items = all * ((int)blockIdx.y + 1) / (int)gridDim.y - first;
    // lanes beyond the items take every sets-th partial result
    const int sets = items >= 256 ? 1 : items > 0 ? 256 / items : 1;
    const int set = (int)threadIdx.x / (items < 256 && items > 0 ? items : 256);
    for (int i0 = 0; i0 < items; i0 += 256) {
        const int i = sets > 1 ? (int)threadIdx.x - set * items : i0 + (int)threadIdx.x;
        const int q = (first + i) / lanes, d = (first + i) % lanes * 4;
        float4 o = make_float4(0, 0, 0, 0);
        float M = kNegInf, L = 0.0f;
        if (i < items && set < sets) {
#pragma unroll 4
            for (int w = w0 + set; w <= w1; w += sets) {
                const float* part = place(p, w, w == w0 ? which0 : 0);
                const float2 ml = *reinterpret_cast<const float2*>(part + 2 * q);
                const float4 x = *reinterpret_cast<const float4*>(part + 32 + q * p.s.dim + d);
                add_part(p.c, M, L, o, ml.x, ml.y, x);
            }
        }
        if (sets > 1) {
            redm[threadIdx.x] = M;
            redl[threadIdx.x] = L;
            red[threadIdx.x] = o;
            for (int n = sets, half; n > 1; n = half) {
                half = (n + 1) / 2;
                __syncthreads();
                if (set < n - half) {
                    const int at = (int)threadIdx.x + half * items;
                    add_part(p.c, M, L, o, redm[at], redl[at], red[at]);
                    redm[threadIdx.x] = M;
                    redl[threadIdx.x] = L;
                    red[threadIdx.x] = o;
                }
            }
        }
        if (set == 0 && i < items) {
            const float inv = 1.0f / L;
            const int64_t at = (int64_t)b * p.a.Hq + head * p.s.group + q0 + q;
            *reinterpret_cast<uint2*>(p.a.out + at * p.s.dim + d) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
            if (p.a.lse && d == 0) p.a.lse[at] = lse_of(p, M, L);
        }
    }
}

// Whether each row stays in one piece, a workgroup to a row: then no join is
// launched (4 to 5 us) and no lengths are scanned, but the longest row is the
// shortest time.  With more rows than workgroups at a time they are taken
// longest first (1024 rows of 128, bf16, random up to 768 tokens 42.0 -> 35.2
// us), up to kSorted sequences.  Split against whole (us; rows of equal length /
// random ones up to it):
//   head_dim 64, e4m3, fp32 queries: 64 rows of 768 tokens 15.6 -> 12.0 / 14.2
//     -> 10.9, of 1024 13.6 -> 15.0; 512 rows of 1024 24.4 -> 18.9 / 19.4 ->
//     16.5, of 2048 34.9 -> 32.4 / 23.6 -> 27.5
//   head_dim 128, bf16: 64 rows of 384 tokens 13.9 -> 11.4, of 768 15.2 -> 16.7;
//     256 rows of 1024 26% / 7% less, of 1536 17% less / 8% more; sorted, 1024
//     rows of 2048 2% / 11% less
// and alike at 192 and 256.  Sorted rows of 2560 tokens and more are level or
// better too, but one long row among short ones would be seen by then.
bool is_whole(int64_t B, int64_t rows, int64_t capacity, int64_t D) {
    int units;
    if (B <= kSorted && rows > kCUs * (D <= 64 ? 3 : 2))
        units = 16;
    else if (rows >= 256)
        units = D <= 64 && rows >= 512 ? 12 : 8;
    else
        units = D <= 64 ? 6 : 3;
    return capacity <= units * kUnit;
}

// per_cu: workgroups per CU at most
Shape shape_of(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages, int per_cu) {
    Shape s;
    s.heads = (int32_t)H;
    s.dim = (int32_t)D;
    s.page_size = (int32_t)page_size;
    s.pg8 = (int32_t)(page_size / 8);
    // g8 / pg8 = umulhi(g8, magic): exact while g8 * pg8 < 2^32.  pg8 == 1
    // would need 2^32; its magic is 0 and look_up adds g8.
    s.magic = s.pg8 == 1 ? 0 : (int32_t)(uint32_t)((uint64_t(1) << 32) / s.pg8 + 1);
    s.group = (int32_t)(Hq / H);
    s.tiles = (s.group + 15) / 16;
    s.rows = s.heads * s.tiles;
    s.capacity = (int32_t)(page_size * max_pages);
    s.whole = is_whole(B, B * s.rows, s.capacity, D);
    const int64_t units = B * s.rows * (s.whole ? 1 : (s.capacity + kUnit - 1) / kUnit + kRowCost);
    // Past 64 columns 4-bit codes' third workgroup per CU may take no more workspace
    // than two with 16 heads, which other types need: its size does not know the type.
    // So a place has only the heads of a tile there, and where those are more than 10
    // there are two.  (16 heads to a key-value head, 64 sequences of up to 16381
    // tokens, 8 heads of 128, with two and three: 133 and 128 us, 32 of up to 8192
    // 41.2 and 40.7, 16 of up to 4099 21.7 and 22.4.)
    const int64_t most = s.whole ? int64_t(1) << 20 : kCUs * (D > 64 && per_cu * heads_of_place(s.dim, s.group) > 32 ? std::min(per_cu, 2) : per_cu);
    s.groups = (int32_t)(units < most ? units : most);
    s.ordered = s.whole && s.capacity > kUnit && B <= kSorted && s.groups == B * s.rows && s.groups > kCUs * per_cu;
    s.by_row = B * s.rows <= s.groups;
    s.crosses = s.by_row ? (int32_t)(B * s.rows) : s.groups;
    return s;
}

size_t workspace_of(const Shape& s, int32_t crosses) {
    return s.whole ? 0 : (size_t)crosses * sizeof(Cross) + (size_t)s.groups * 2 * numbers_of_place(s.dim, s.group) * sizeof(float);
}

}  // namespace

size_t attend_workspace_bytes(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages) {
    // the size does not know the types: as for those that take the most workgroups
    int most = 1;
    for (const int held : {BD_BF16, BD_E4M3, BD_E2M1})
        for (int split_q = 0; split_q < 2; ++split_q) {
            const int n = per_cu(width_of((int)D, held), split_q, held);
            most = n > most ? n : most;
        }
    const Shape s = shape_of(B, Hq, H, D, page_size, max_pages, most);
    return workspace_of(s, s.groups);  // the table never has more entries
}

hipError_t launch_attend(const AttendArgs& a, bool q_fp32, hipStream_t stream) {
    const int held = a.kv.type, D = a.kv.head_dim;
    const bool formed = a.cap > 0.0f || a.slopes || a.first;
    const auto unit16 = [&](int64_t stride) { return (uint32_t)(stride * (held == BD_BF16 ? 2 : 1) / 16); };
    const uint32_t head_scales = (uint32_t)(a.kv.page_size * (held == BD_E2M1 ? D / kGroup4 : 1));
    const float scale = __builtin_fabsf(a.scale);
    const Form form = form_of(a.scale, a.cap);
    Args p{a, shape_of(a.B, a.Hq, a.kv.num_heads, D, a.kv.page_size, a.max_pages,
                     per_cu(width_of(D, held), q_fp32, held)),
           (uint32_t)a.kv.num_pages, unit16(a.kv.page_stride), unit16(a.kv.head_stride), unit16(a.kv.token_stride),
           a.kv.num_heads * head_scales, head_scales,
           __builtin_fmaxf((formed ? form.unit : scale) * 1.4426950408889634f, kLeastC),
           formed ? form.unit : scale, form.times, a.scale < 0.0f ? 0x80008000u : 0u};
    if (workspace_of(p.s, p.s.crosses) > attend_workspace_bytes(a.B, a.Hq, a.kv.num_heads, D, a.kv.page_size, a.max_pages))
        return hipErrorInvalidValue;  // what is laid out here is what the caller was told to bring
    if (held == BD_E2M1)
        formed ? go_e2m1_formed(p, q_fp32, stream) : go_e2m1(p, q_fp32, stream);
    else if (held == BD_E4M3)
        formed ? go_e4m3_formed(p, q_fp32, stream) : go_e4m3(p, q_fp32, stream);
    else
        formed ? go_bf16_formed(p, q_fp32, stream) : go_bf16(p, q_fp32, stream);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.s.whole) return e;
    // about two workgroups per CU: a row's items, 8 or more, on as many as that leaves
    const int most = (p.s.group < 16 ? p.s.group : 16) * D / 32;
    const int per = 2 * kCUs / p.s.crosses;
    const int y = most < per ? most : per;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)p.s.crosses, (unsigned)(y < 1 ? 1 : y)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace bd
