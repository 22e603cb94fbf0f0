// Attention of a prompt's tokens: how a launch is split, its dispatch, and the
// join of split rows.  The kernel and what bounds it: prompt_device.h.
#include "prompt_device.h"

namespace bd {
using namespace prompt;
namespace {

// A tile's rows of one head: the sum of its splits' partial outputs over the sum
// of their sums, each scaled to the common maximum, in order.  Four values of a
// row to a lane.
__global__ __launch_bounds__(256) void join_kernel(const Args p) {
    const int head = blockIdx.x % p.heads, from_end = blockIdx.x / p.heads;
    const Tile tile = tile_at(p, from_end);
    if (tile.none) return;
    const int given = tile.given;
    const int len = given > p.capacity || given < 0 ? 0 : given;
    const int lanes = p.dim / 4;
    const int rows = tile.n * p.group - tile.row < p.rows ? tile.n * p.group - tile.row : p.rows;
    const int items = rows * lanes;
    for (int i = (int)(blockIdx.y * 256 + threadIdx.x); i < items; i += (int)gridDim.y * 256) {
        const int r = i / lanes, d = (i - r * lanes) * 4;
        const int token = (tile.row + r) / p.group, qhead = head * p.group + (tile.row + r) - token * p.group;
        float M = kNegInf, L = 0.0f;
        float4 o = make_float4(0, 0, 0, 0);
#pragma unroll 4
        for (int s = 0; s < p.splits; ++s) {
            const float* part = place(p, from_end, head, s);
            const float m = part[2 * r], l = part[2 * r + 1];
            const float4 x = *reinterpret_cast<const float4*>(part + 2 * p.rows + r * p.dim + d);
            // a part whose scores are all -infinity, or that saw no keys, has sum and output 0 (or NaN)
            const float to = fmaxf(M, m);
            const float f = M == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((M - to) * p.c);
            const float g = m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((m - to) * p.c);
            M = to;
            L = L * f + l * g;
            o.x = o.x * f + x.x * g, o.y = o.y * f + x.y * g, o.z = o.z * f + x.z * g, o.w = o.w * f + x.w * g;
        }
        const Range range = range_of(p, tile, len, token);
        const bool sees = range.hi > range.lo;
        float inv = sees ? 1.0f / L : 0.0f;
        if (given > p.capacity) inv = __builtin_nanf("");
        const int64_t at = (int64_t)(tile.start + token) * p.a.Hq + qhead;
        *reinterpret_cast<uint2*>(p.a.out + at * p.dim + d) =
            make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
        if (p.a.lse && d == 0) {
            const float v = __builtin_fmaf(M, p.unit, __builtin_amdgcn_logf(L) * 0.69314718055994531f);
            p.a.lse[at] = given > p.capacity ? __builtin_nanf("") : sees ? v : kNegInf;
        }
    }
}

// Tiles at most: whole ones of all rows, and one that is not for each sequence.
int64_t tiles_at_most(int64_t T, int64_t B, int64_t group, int rows) { return T * group / rows + B; }
int rows_of(int64_t D, int held, bool form) { return 32 * waves_of(width_of((int)D), held, form); }

// Workgroups that share a tile's keys.  `places` of them run at a time: two of 4
// waves on each CU, or one of 8 or of 256 columns.  A split costs what its keys
// do, a start and an end of about 256 keys, and where there are several the
// partial results (350 more, and 250 for the join's launch); what is least is
// taken of 1 and the numbers that fill 1 to 4 rounds of places, while each has
// 256 keys of a full table.  The sequences are taken to be alike, as the host
// does not know them.  (us with 1 workgroup / those that fill a round / one more
// for each tile, bf16, 64 heads of 128 over 8: 3 sequences of 5 tokens behind
// 16000 - / 41 / 48, 32 of them 331 / 232 / -; 300 tokens behind 8192 - / 101 /
// 128; 512 tokens of their own 23 / 29 / -.)
int64_t splits_of(int64_t T, int64_t B, int64_t group, int64_t heads, int64_t capacity, int64_t D, int rows) {
    if (T < 1 || B < 1) return 1;
    const int64_t groups = B * (((T + B - 1) / B * group + rows - 1) / rows) * heads;
    const int64_t places = rows == 128 && D <= 192 ? 512 : 256;
    const int64_t most = capacity / 256;
    int64_t best = 1, least = (groups + places - 1) / places * (capacity + 256);
    for (int r = 1; r <= 4; ++r) {
        int64_t n = r * places / groups;
        n = n < most ? n : most;
        if (n < 2) continue;
        const int64_t cost = (groups * n + places - 1) / places * (capacity / n + 256 + 350) + 250;
        if (cost < least) best = n, least = cost;
    }
    return best;
}

}  // namespace

// Enough for every type of cache, whose tiles have one number of rows or the other.
size_t prompt_workspace_bytes(int64_t T, int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t capacity) {
    size_t bytes = 0;
    for (const int held : {BD_BF16, BD_E4M3}) {
        const int rows = rows_of(D, held, false);
        const int64_t tiles = tiles_at_most(T, B, Hq / H, rows), splits = splits_of(T, B, Hq / H, H, capacity, D, rows);
        const size_t n = splits == 1 ? 0 : (size_t)(tiles * H * splits * rows * (D + 2)) * sizeof(float);
        bytes = n > bytes ? n : bytes;
    }
    return bytes;
}

hipError_t launch_prompt(const PromptArgs& a, hipStream_t stream) {
    const int held = a.kv.type, D = a.kv.head_dim, H = a.kv.num_heads;
    const bool formed = a.cap > 0.0f || a.slopes;
    const auto unit16 = [&](int64_t stride) { return (uint32_t)(stride * (held == BD_BF16 ? 2 : 1) / 16); };
    const uint32_t head_scales = (uint32_t)(a.kv.page_size * (held == BD_E2M1 ? D / kGroup4 : 1));
    const float scale = __builtin_fabsf(a.scale);
    const Form form = form_of(a.scale, a.cap);
    const int pg8 = a.kv.page_size / 8;
    const int rows = rows_of(D, held, formed);
    const int64_t tiles = tiles_at_most(a.T, a.B, a.Hq / H, rows);
    const Args p{a, D, H, a.Hq / H, rows, pg8, pg8 == 1 ? 0 : (int32_t)(uint32_t)((uint64_t(1) << 32) / pg8 + 1),
                 a.kv.page_size * a.max_pages, (int32_t)splits_of(a.T, a.B, a.Hq / H, H, (int64_t)a.kv.page_size * a.max_pages, D, rows),
                 (uint32_t)a.kv.num_pages, unit16(a.kv.page_stride), unit16(a.kv.head_stride),
                 unit16(a.kv.token_stride), H * head_scales, head_scales,
                 __builtin_fmaxf((formed ? form.unit : scale) * 1.4426950408889634f, kLeastC),
                 formed ? form.unit : scale, form.times, a.scale < 0.0f ? 0x80008000u : 0u};
    const unsigned groups = (unsigned)(tiles * H * p.splits);
    if (held == BD_E2M1)
        formed ? go_e2m1_formed(p, groups, stream) : go_e2m1(p, groups, stream);
    else if (held == BD_E4M3)
        formed ? go_e4m3_formed(p, groups, stream) : go_e4m3(p, groups, stream);
    else
        formed ? go_bf16_formed(p, groups, stream) : go_bf16(p, groups, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    // the rows of a tile over as many workgroups as make about four for each CU
    int64_t y = 4 * 256 / (tiles * H);
    const int64_t most = (int64_t)rows * D / 4 / 256;
    y = y < 1 ? 1 : y > most ? most : y;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)(tiles * H), (unsigned)y), dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace bd
