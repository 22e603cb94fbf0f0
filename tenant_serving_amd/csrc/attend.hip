// Attention of one new token per sequence over the paged key-value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c q.k_j - m),  c = scale log2(e)
//
// with m the running maximum of c q.k_j: one pass over the cache, which is
// read exactly once, so the kernel is bound by HBM.
//
// Layout.  The query heads that share a key-value head (up to 16 of them) are
// the 16 columns of v_mfma_f32_16x16x32_bf16; a wave takes 32 tokens at a
// time and nothing passes through LDS on the way:
//   scores  S^T [tokens, heads] = K Q^T.  A lane's A operand is 8 consecutive
//           values of one key row, a 16-byte load (e4m3 codes are converted
//           in registers).  Two 16-token products cover the tile; their rows
//           are the tokens 8 (r / 4) + r % 4 and those + 4, which leaves each
//           lane with the scores of 8 consecutive tokens 8 g .. 8 g + 7 of one
//           head (g = lane / 16),
//   sums    O^T [dims, heads] += V^T P^T, whose B operand is just those 8
//           tokens, so the weights stay in their lane.  The A operand needs 8
//           tokens of one value column: a lane loads its piece of 8 value
//           rows (16 bytes at head_dim 128) and pairs them up with byte
//           permutes, one per two values.
// The running maximum moves only when a score passes it by 2^10, which one
// compare and a ballot find out: then the wave exchanges maxima and rescales.
// The weights enter as two bf16 terms (their sum holds 16 bits), and so do
// fp32 queries: the matrix units idle most of the time here, and an output
// is then as exact as its own rounding.
//
// Work split.  A unit is 128 tokens of one (sequence, key-value head, 16
// query heads), four waves with a tile each.  The units of the whole batch
// lie in one line, which the workgroups share out evenly, whatever the
// lengths: every workgroup works the line up from the device's lengths by
// itself.  A row of units that ends up in several workgroups leaves fp32
// partial results (sum, maximum, unnormalised output) in the workspace, and
// join_kernel adds them in workgroup order.
#include "step_internal.h"

namespace bd {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 32;                  // tokens of a wave
constexpr int kUnit = kWaves * kTile;      // tokens of a unit
constexpr int kGroups = 512;               // workgroups at most: two per CU
constexpr float kLazy = 10.0f;             // log2: how far a score may pass the running maximum
constexpr float kNegInf = -__builtin_inff();

struct Shape {
    int32_t heads, dim, page_size, pg8, magic;  // pg8: groups of 8 tokens in a page
    int32_t group, tiles;                       // query heads per kv head, and tiles of 16 of them
    int32_t rows;                               // rows of units per sequence: heads * tiles
    int32_t capacity, groups;                   // tokens a table row holds; workgroups launched
    int32_t crosses, by_row;                    // entries of the workspace's table
};

struct Args {
    AttendArgs a;
    Shape s;
    float c;  // scale * log2(e)
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Units of one row of a sequence: at least one, so that an empty sequence's
// outputs are written too; one where the length is out of range.
__device__ __forceinline__ int units_of(int len, int capacity) {
    return len <= kUnit || len > capacity ? 1 : (len + kUnit - 1) / kUnit;
}

// The batch's line of units, worked out by each wave: lane l sums the
// sequences [l n, l n + n).
struct Line {
    int n, first, total;  // per lane: sequences, units before its own; units of the batch
    __device__ __forceinline__ void scan(const Args& p) {
        const int lane = threadIdx.x & 63;
        n = (p.a.B + 63) / 64;
        int sum = 0;
        const int b0 = lane * n;
        for (int i = 0; i < n; ++i)
            if (b0 + i < p.a.B) sum += units_of(p.a.lengths[b0 + i], p.s.capacity);
        sum *= p.s.rows;
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        first = inc - sum;
        total = __shfl(inc, 63, 64);
    }
    // The sequence that holds unit u, and its first unit.
    __device__ __forceinline__ int holder_of(const Args& p, int u, int* start) const {
        const int lane = threadIdx.x & 63;
        // the last lane that has sequences and starts at or before u
        const uint64_t at = __ballot(lane * n < p.a.B && first <= u);
        const int l = 63 - __clzll(at);
        int s = uni(__shfl(first, l, 64));
        int b = l * n;
        for (;;) {
            const int len = units_of(p.a.lengths[b], p.s.capacity) * p.s.rows;
            if (u < s + len || b + 1 >= p.a.B) break;
            s += len;
            ++b;
        }
        *start = uni(s);
        return uni(b);
    }
};

// Workgroup w of W takes the units [start(w), start(w + 1)).
struct Cut {
    int W, q, r;
    __device__ __forceinline__ Cut(int total, int groups) {
        W = total < groups ? total : groups;
        q = total / W;
        r = total - q * W;
    }
    __device__ __forceinline__ int start(int w) const { return w * q + (w < r ? w : r); }
    __device__ __forceinline__ int group_of(int u) const {
        const int big = r * (q + 1);
        return u < big ? u / (q + 1) : r + (u - big) / q;
    }
};

// The workspace: a table of Cross, then each workgroup's partial results, two
// places (the first row it works on and the last one) of 16 heads' (maximum,
// sum) and unnormalised outputs.
//
// Cross: a row of units that starts in one workgroup and goes on in the next
// ones.  The table has an entry per row of the batch where these are fewer
// than the workgroups, else one per workgroup (in which at most one such row
// starts); each is written in every call.
struct Cross {
    int32_t at;     // b * rows + row
    int32_t first;  // the workgroup it starts in, times 2, plus its place there; -1: all of it is in one workgroup
    int32_t last;   // the workgroup it ends in
    int32_t pad;
};
__device__ __forceinline__ float* place(const Args& p, int w, int which) {
    return p.a.part + (int64_t)p.s.crosses * 4 + ((int64_t)w * 2 + which) * (16 * (p.s.dim + 2));
}

// Page lookups: token group g8 (8 tokens, which no page boundary cuts) of a
// sequence lies in page table[g8 / pg8].
struct Where {
    int64_t at;  // element of the group's first token in the cache's arrays
    int64_t sc;  // its scale byte
    bool bad;
};
__device__ __forceinline__ int page_index(const Shape& s, int g8) {
    // exact: g8 < 2^21, pg8 <= 2^9
    return (int)__umulhi((uint32_t)g8, (uint32_t)s.magic) + (s.pg8 == 1 ? g8 : 0);
}
__device__ __forceinline__ Where locate(const Args& p, int g8, int idx, int page, int head) {
    Where w;
    w.bad = page < 0 || page >= p.a.kv.num_pages;
    page = w.bad ? 0 : page;
    const int at = (g8 - idx * p.s.pg8) * 8;
    w.at = page * p.a.kv.page_stride + head * p.a.kv.head_stride + at * p.a.kv.token_stride;
    w.sc = ((int64_t)page * p.s.heads + head) * p.s.page_size + at;
    return w;
}

template <int N>
struct Dwords {
    uint32_t d[N];
};
// The cache is read once: streaming loads (against plain ones, 64 sequences of
// 8192 tokens in e4m3 187 -> 173 us, 4 of 131072 in bf16 365 -> 334).
template <int N>
__device__ __forceinline__ Dwords<N> load_dwords(const void* p) {
    Dwords<N> r;
    if constexpr (N == 1) {
        r.d[0] = *static_cast<const uint32_t*>(p);  // rows of half a cache line, whose other half comes next
    } else if constexpr (N == 2) {
        typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
        const u32x2_t v = __builtin_nontemporal_load(static_cast<const u32x2_t*>(p));
        r.d[0] = v.x, r.d[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const uint4 v = load_stream16(static_cast<const uint4*>(p) + i);
            r.d[4 * i] = v.x, r.d[4 * i + 1] = v.y, r.d[4 * i + 2] = v.z, r.d[4 * i + 3] = v.w;
        }
    }
    return r;
}
template <int N>
__device__ __forceinline__ void clear(Dwords<N>& r) {
#pragma unroll
    for (int i = 0; i < N; ++i) r.d[i] = 0;
}

// kDC: head_dim rounded up to 64, 128 or 256.  kFull: head_dim is kDC.
// kSplitQ: fp32 queries as two bf16 terms.
template <int kDC, bool kFull, bool kE4m3, bool kSplitQ>
__global__ __launch_bounds__(kWaves * 64, kDC == 256 ? 1 : 2) void attend_kernel(const Args p) {
    constexpr int NS = kDC / 32;              // k-steps of a score product
    constexpr int DV = kDC / 16;              // value columns of a lane
    constexpr int KL = kE4m3 ? NS / 2 : NS;   // 16-byte loads of a key row per lane
    constexpr int VD = kE4m3 ? DV / 4 : DV / 2;  // dwords of a value row per lane
    constexpr int kPad = kDC + 4;
    __shared__ float so[kWaves][16][kPad];
    __shared__ float sm[kWaves][16], sl[kWaves][16];

    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    Line line;
    line.scan(p);
    const Cut cut(line.total, p.s.groups);
    const int w = blockIdx.x;
    Cross* crosses = reinterpret_cast<Cross*>(p.a.part);
    const bool by_row = p.s.by_row;
    if (!by_row && crosses && threadIdx.x == 0) crosses[w].first = -1;
    if (w >= cut.W) return;
    int u = cut.start(w);
    const int end = cut.start(w + 1);
    int seq_start;
    int b = line.holder_of(p, u, &seq_start);
    int len = uni(p.a.lengths[b]);
    int un = units_of(len, p.s.capacity);
    int row = (u - seq_start) / un;
    int unit = u - seq_start - row * un;
    bool first_row = true;

    while (u < end) {
        const int n = un - unit < end - u ? un - unit : end - u;
        const int head = row / p.s.tiles;
        const int q0 = (row - head * p.s.tiles) * 16;  // the tile's first query head of the group
        const int nq = p.s.group - q0 < 16 ? p.s.group - q0 : 16;
        const int hq0 = head * p.s.group + q0;
        const bool too_long = len > p.s.capacity;
        const int tokens = too_long || len < 0 ? 0 : len;
        const int stop = tokens < (unit + n) * kUnit ? tokens : (unit + n) * kUnit;

        // queries: B operand, column i16, k = the head's values in the order
        // in which the key loads bring them
        uint4 qh[NS], ql[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int d = kE4m3 ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
            float f[8];
            Raw8<kSplitQ> raw;
            raw.zero();
            if (i16 < nq && (kFull || d < p.s.dim)) raw.load(p.a.q, b * p.a.qs.token + (hq0 + i16) * p.a.qs.head + d);
            raw.widen(f);
            qh[s] = narrow_bf16x8(f);
            if (kSplitQ) {
                float back[8];
                widen_bf16x8(qh[s], back);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] -= back[j];
                ql[s] = narrow_bf16x8(f);
            }
        }

        f32x4_t acc[DV];
        float m, mm, l;  // mm: m, or 0 while m is -infinity
        bool bad = false;
        float c = p.c;
        int pass = 0;  // 1: again, see below
        bool lost = false;

        const int32_t* table = p.a.table + b * p.a.table_stride;
        const int last8 = tokens > 0 ? (tokens - 1) >> 3 : 0;
        const int t0 = unit * kUnit + wave * kTile;

        // A tile's loads, in flight while the tile before it is worked on:
        // the page numbers a tile earlier, the keys as soon as the scores are
        // done with the registers, the values after the sums.
        Dwords<4> kk[2][KL];
        Dwords<VD> vv[8];
        float ks[2];
        uint2 vs;
        int pk, pv;  // page numbers of the lane's key rows and value rows
        const auto group_of = [&](int t, int add) {
            const int g8 = (t >> 3) + add;
            return g8 < last8 ? g8 : last8;
        };
        const auto load_pages = [&](int t) {
            pk = table[page_index(p.s, group_of(t, i16 >> 2))];
            pv = table[page_index(p.s, group_of(t, g))];
        };
        const auto load_keys = [&](int t) {
            const int g8 = group_of(t, i16 >> 2);
            const Where w = locate(p, g8, page_index(p.s, g8), pk, head);
            bad |= w.bad;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = w.at + ((i16 & 3) + 4 * h) * p.a.kv.token_stride;
#pragma unroll
                for (int s = 0; s < KL; ++s) {
                    const int d = kE4m3 ? s * 64 + g * 16 : s * 32 + g * 8;
                    clear(kk[h][s]);
                    if (kFull || d < p.s.dim)
                        kk[h][s] = load_dwords<4>(static_cast<const char*>(p.a.kv.k) + (at + d) * (kE4m3 ? 1 : 2));
                }
                if (kE4m3) ks[h] = scale_of(p.a.kv.k_scales[w.sc + (i16 & 3) + 4 * h]);
            }
        };
        const auto load_values = [&](int t) {
            const int g8 = group_of(t, g);
            const Where w = locate(p, g8, page_index(p.s, g8), pv, head);
            bad |= w.bad;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                clear(vv[j]);
                if (kFull || i16 * DV < p.s.dim)
                    vv[j] = load_dwords<VD>(static_cast<const char*>(p.a.kv.v) +
                                            (w.at + j * p.a.kv.token_stride + i16 * DV) * (kE4m3 ? 1 : 2));
            }
            if (kE4m3) vs = *reinterpret_cast<const uint2*>(p.a.kv.v_scales + w.sc);
        };

    again:
#pragma unroll
        for (int j = 0; j < DV; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        m = kNegInf, mm = 0.0f, l = 0.0f;
        if (t0 < stop) {
            load_pages(t0);
            load_keys(t0);
            load_values(t0);
            load_pages(t0 + kUnit);  // past the end: the last group's page
        }
#pragma nounroll
        for (int t = t0; t < stop; t += kUnit) {
            const bool more = t + kUnit < stop;
            // scores of tokens t + 8 g + j, head i16
            float sc[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                f32x4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    uint4 kb;
                    if constexpr (kE4m3) {
                        const uint32_t c0 = kk[h][s / 2].d[2 * (s & 1)], c1 = kk[h][s / 2].d[2 * (s & 1) + 1];
                        kb = make_uint4(e4m3x2_to_bf16<false>(c0, ks[h]), e4m3x2_to_bf16<true>(c0, ks[h]),
                                        e4m3x2_to_bf16<false>(c1, ks[h]), e4m3x2_to_bf16<true>(c1, ks[h]));
                    } else {
                        const Dwords<4>& r = kk[h][s];
                        kb = make_uint4(r.d[0], r.d[1], r.d[2], r.d[3]);
                    }
                    if (kSplitQ) x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(kb), as_bf16x8(ql[s]), x, 0, 0, 0);
                    x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(kb), as_bf16x8(qh[s]), x, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[4 * h + r] = x[r] * c;
            }
            if (more) load_keys(t + kUnit);
            const bool tail = t + kTile > tokens;
            if (tail) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool out = t + 8 * g + j >= tokens;
                    sc[j] = out ? kNegInf : sc[j];
#pragma unroll
                    for (int i = 0; i < VD; ++i) vv[j].d[i] = out ? 0u : vv[j].d[i];
                    if constexpr (kE4m3) {  // any byte may stand there: 2^0
                        uint32_t& sw = j < 4 ? vs.x : vs.y;
                        const uint32_t field = 0xffu << (8 * (j & 3));
                        sw = out ? (sw & ~field) | (127u << (8 * (j & 3))) : sw;
                    }
                }
            }

            float mx = sc[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) mx = fmaxf(mx, sc[j]);
            if (__ballot(mx > m + kLazy)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                const float up = fmaxf(m, mx);
                const float to = up == kNegInf ? 0.0f : up;
                const float f = __builtin_amdgcn_exp2f(m - to);
                m = up;
                mm = to;
                l *= f;
#pragma unroll
                for (int j = 0; j < DV; ++j) acc[j] *= f;
            }
            float pr[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                pr[j] = __builtin_amdgcn_exp2f(sc[j] - mm);
                l += pr[j];
            }
            const uint4 ph = narrow_bf16x8(pr);
            float back[8];
            widen_bf16x8(ph, back);
#pragma unroll
            for (int j = 0; j < 8; ++j) back[j] = pr[j] - back[j];
            uint4 pl = narrow_bf16x8(back);
            if (pass) pl = ph;

            // value rows as bf16 pairs of columns, then pairs of tokens
            uint32_t vb[8][DV / 2];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (kE4m3) {
                    const uint32_t sw = j < 4 ? vs.x : vs.y;
                    const float s = scale_of((sw >> (8 * (j & 3))) & 0xff);
#pragma unroll
                    for (int i = 0; i < VD; ++i) {
                        vb[j][2 * i] = e4m3x2_to_bf16<false>(vv[j].d[i], s);
                        vb[j][2 * i + 1] = e4m3x2_to_bf16<true>(vv[j].d[i], s);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < DV / 2; ++i) vb[j][i] = vv[j].d[i];
                }
            }
#pragma unroll
            for (int j = 0; j < DV; ++j) {
                uint32_t va[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    va[i] = __builtin_amdgcn_perm(vb[2 * i + 1][j / 2], vb[2 * i][j / 2],
                                                  j & 1 ? 0x07060302u : 0x05040100u);
                const bf16x8_t av = as_bf16x8(make_uint4(va[0], va[1], va[2], va[3]));
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, as_bf16x8(pl), acc[j], 0, 0, 0);
                acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, as_bf16x8(ph), acc[j], 0, 0, 0);
            }
            if (more) {
                load_values(t + kUnit);
                load_pages(t + 2 * kUnit);
            }
        }

        // A second term breaks on infinities: it is of either sign or zero,
        // and infinity minus itself or times zero is NaN.  So where a sum is
        // not finite the wave goes over its tokens again with one term, taken
        // twice and halved, and takes what was lost from there.  The queries'
        // second term only goes where the scores broke.
        if (!pass) {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < DV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) z = __builtin_fmaf(acc[j][r], 0.0f, z);
            if (__ballot(i16 < nq && (z != 0.0f || l != l))) {
                lost = kSplitQ && __ballot(i16 < nq && l != l);
                float* keep = &so[wave][0][0] + lane;
#pragma unroll
                for (int j = 0; j < DV; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) keep[(4 * j + r) * 64] = acc[j][r];
                if (lost) {
#pragma unroll
                    for (int s = 0; s < NS; ++s) ql[s] = qh[s];
                    c *= 0.5f;
                }
                pass = 1;
                goto again;
            }
        } else {
            const float* keep = &so[wave][0][0] + lane;
#pragma unroll
            for (int j = 0; j < DV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = keep[(4 * j + r) * 64];
                    acc[j][r] = !lost && x * 0.0f == 0.0f ? x : acc[j][r] * 0.5f;
                }
        }

        // the wave's result, then the workgroup's: heads i16, values
        // (4 g + r) DV + j of acc[j][r]
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (__ballot(bad) || too_long) l = __builtin_nanf("");
        if (lane < 16) sm[wave][i16] = m, sl[wave][i16] = l;
        __syncthreads();
        float top = sm[0][i16];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) top = fmaxf(top, sm[v][i16]);
        const float f = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        if (i16 < nq) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < DV; j += 4) {
                    float4 o = make_float4(acc[j][r] * f, acc[j + 1][r] * f, acc[j + 2][r] * f, acc[j + 3][r] * f);
                    *reinterpret_cast<float4*>(&so[wave][i16][(4 * g + r) * DV + j]) = o;
                }
        }
        __syncthreads();

        const bool whole = n == un;
        const int d4 = p.s.dim / 4;
        float* part = whole ? nullptr : place(p, w, first_row ? 0 : 1);
        if (unit == 0 && crosses && threadIdx.x == 0 && (by_row || !whole)) {
            const int at = b * p.s.rows + row;
            crosses[by_row ? at : w] = Cross{at, whole ? -1 : w * 2 + (first_row ? 0 : 1), cut.group_of(u + un - 1), 0};
        }
        for (int i = threadIdx.x; i < nq * d4; i += kWaves * 64) {
            const int q = i / d4, d = (i - q * d4) * 4;
            float M = sm[0][q];
#pragma unroll
            for (int v = 1; v < kWaves; ++v) M = fmaxf(M, sm[v][q]);
            float L = 0.0f;
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                // a wave without tokens has sum 0 (or NaN where a page was bad)
                L += sl[v][q] * (sm[v][q] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(sm[v][q] - M));
                const float4 x = *reinterpret_cast<const float4*>(&so[v][q][d]);
                o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
            }
            if (whole) {
                const float inv = len <= 0 ? 0.0f : 1.0f / L;
                const int64_t at = (int64_t)b * p.a.Hq + hq0 + q;
                *reinterpret_cast<uint2*>(p.a.out + at * p.s.dim + d) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (p.a.lse && d == 0) p.a.lse[at] = len <= 0 ? kNegInf : (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
            } else {
                *reinterpret_cast<float4*>(part + 32 + q * p.s.dim + d) = o;
                if (d == 0) part[2 * q] = M, part[2 * q + 1] = L;
            }
        }
        first_row = false;
        u += n;
        unit = 0;
        if (u < end && ++row == p.s.rows) {
            row = 0;
            ++b;
            len = uni(p.a.lengths[b]);
            un = units_of(len, p.s.capacity);
        }
        __syncthreads();
    }
}

// Adds a partial result (maximum m, sum l, unnormalised output x) to a running
// one.  A part whose scores are all -infinity has sum and output 0 (or NaN).
__device__ __forceinline__ void add_part(float& M, float& L, float4& o, float m, float l, float4 x) {
    const float to = fmaxf(M, m);
    const float f = M == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(M - to);
    const float g = m == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m - to);
    M = to;
    L = L * f + l * g;
    o.x = o.x * f + x.x * g, o.y = o.y * f + x.y * g, o.z = o.z * f + x.z * g, o.w = o.w * f + x.w * g;
}

// Rows of units that several workgroups worked on: out = sum of their partial
// outputs over the sum of their sums, each scaled to the common maximum.  The
// heads of a row are shared out over grid y.
__global__ __launch_bounds__(256) void join_kernel(const Args p) {
    __shared__ float4 red[256];
    __shared__ float redm[256], redl[256];
    const Cross cross = reinterpret_cast<const Cross*>(p.a.part)[blockIdx.x];
    if (cross.first < 0) return;
    const int w0 = cross.first >> 1, w1 = cross.last, which0 = cross.first & 1;
    const int b = cross.at / p.s.rows, row = cross.at - b * p.s.rows;
    const int head = row / p.s.tiles, q0 = (row - head * p.s.tiles) * 16;
    const int nq = p.s.group - q0 < 16 ? p.s.group - q0 : 16;
    // this workgroup's heads, and its work: 4 values of one head per item
    const int qa = nq * (int)blockIdx.y / (int)gridDim.y, qe = nq * ((int)blockIdx.y + 1) / (int)gridDim.y;
    const int lanes = p.s.dim / 4, items = (qe - qa) * lanes;
    // lanes beyond the items take every sets-th partial result
    const int sets = items >= 256 ? 1 : items > 0 ? 256 / items : 1;
    const int set = (int)threadIdx.x / (items < 256 && items > 0 ? items : 256);
    for (int i0 = 0; i0 < items; i0 += 256) {
        const int i = sets > 1 ? (int)threadIdx.x - set * items : i0 + (int)threadIdx.x;
        const int q = qa + i / lanes, d = i % lanes * 4;
        float4 o = make_float4(0, 0, 0, 0);
        float M = kNegInf, L = 0.0f;
        if (i < items && set < sets) {
#pragma unroll 4
            for (int w = w0 + set; w <= w1; w += sets) {
                const float* part = place(p, w, w == w0 ? which0 : 0);
                const float2 ml = *reinterpret_cast<const float2*>(part + 2 * q);
                const float4 x = *reinterpret_cast<const float4*>(part + 32 + q * p.s.dim + d);
                add_part(M, L, o, ml.x, ml.y, x);
            }
        }
        if (sets > 1) {
            redm[threadIdx.x] = M;
            redl[threadIdx.x] = L;
            red[threadIdx.x] = o;
            __syncthreads();
            if (set == 0)
                for (int k = 1; k < sets; ++k) {
                    const int at = k * items + (int)threadIdx.x;
                    add_part(M, L, o, redm[at], redl[at], red[at]);
                }
        }
        if (set == 0 && i < items) {
            const float inv = 1.0f / L;
            const int64_t at = (int64_t)b * p.a.Hq + head * p.s.group + q0 + q;
            *reinterpret_cast<uint2*>(p.a.out + at * p.s.dim + d) =
                make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
            if (p.a.lse && d == 0) p.a.lse[at] = (M + __builtin_amdgcn_logf(L)) * 0.69314718055994531f;
        }
    }
}

Shape shape_of(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages) {
    Shape s;
    s.heads = (int32_t)H;
    s.dim = (int32_t)D;
    s.page_size = (int32_t)page_size;
    s.pg8 = (int32_t)(page_size / 8);
    // g8 / pg8 = umulhi(g8, magic): exact while g8 * pg8 < 2^32.  pg8 == 1
    // would need 2^32; its magic is 0 and page_index adds g8.
    s.magic = s.pg8 == 1 ? 0 : (int32_t)(uint32_t)((uint64_t(1) << 32) / s.pg8 + 1);
    s.group = (int32_t)(Hq / H);
    s.tiles = (s.group + 15) / 16;
    s.rows = s.heads * s.tiles;
    s.capacity = (int32_t)(page_size * max_pages);
    const int64_t per_row = s.capacity <= kUnit ? 1 : (s.capacity + kUnit - 1) / kUnit;
    const int64_t units = B * s.rows * per_row;
    // a capacity of one unit splits nothing: a workgroup per row of units
    const int64_t most = per_row == 1 ? int64_t(1) << 20 : kGroups;
    s.groups = (int32_t)(units < most ? units : most);
    s.by_row = B * s.rows <= s.groups;
    s.crosses = s.by_row ? (int32_t)(B * s.rows) : s.groups;
    return s;
}

template <int kDC, bool kFull>
void go(const Args& p, bool q_fp32, hipStream_t s) {
    const dim3 grid((unsigned)p.s.groups), block(kWaves * 64);
    if (p.a.kv.type == BD_E4M3) {
        if (q_fp32)
            hipLaunchKernelGGL((attend_kernel<kDC, kFull, true, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((attend_kernel<kDC, kFull, true, false>), grid, block, 0, s, p);
    } else {
        if (q_fp32)
            hipLaunchKernelGGL((attend_kernel<kDC, kFull, false, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((attend_kernel<kDC, kFull, false, false>), grid, block, 0, s, p);
    }
}

}  // namespace

size_t attend_workspace_bytes(int64_t B, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t max_pages) {
    if (page_size * max_pages <= kUnit) return 0;
    const Shape s = shape_of(B, Hq, H, D, page_size, max_pages);
    return (size_t)s.crosses * sizeof(Cross) + (size_t)s.groups * 2 * 16 * (D + 2) * sizeof(float);
}

hipError_t launch_attend(const AttendArgs& a, bool q_fp32, hipStream_t stream) {
    Args p{a, shape_of(a.B, a.Hq, a.kv.num_heads, a.kv.head_dim, a.kv.page_size, a.max_pages),
           a.scale * 1.4426950408889634f};
    const int D = a.kv.head_dim;
    if (D <= 64) {
        if (D == 64)
            go<64, true>(p, q_fp32, stream);
        else
            go<64, false>(p, q_fp32, stream);
    } else if (D <= 128) {
        if (D == 128)
            go<128, true>(p, q_fp32, stream);
        else
            go<128, false>(p, q_fp32, stream);
    } else {
        if (D == 256)
            go<256, true>(p, q_fp32, stream);
        else
            go<256, false>(p, q_fp32, stream);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.s.capacity <= kUnit) return e;
    // about two workgroups per CU: a row's heads on as many as that leaves
    const int nq = p.s.group < 16 ? p.s.group : 16;
    const int per = kGroups / p.s.crosses < 1 ? 1 : kGroups / p.s.crosses;
    hipLaunchKernelGGL(join_kernel, dim3((unsigned)p.s.crosses, (unsigned)(nq < per ? nq : per)), dim3(256), 0, stream,
                       p);
    return hipGetLastError();
}

}  // namespace bd
