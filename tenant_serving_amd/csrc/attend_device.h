// Attention of one new token per sequence over the paged key-value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (q.k_j - m)),  c = scale log2(e)
//
// with m the running maximum of q.k_j: one pass over the cache for each 16
// query heads that share a key-value head, bound by HBM.
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
// The running maximum moves only when a weight would pass 2^10, which one
// compare and a ballot find out: then the wave exchanges maxima and rescales.
// It is kept as a score, without c: the difference is taken first, so that the
// largest score's weight is 2^0 however large the scores are (2^(c q.k_j - c m)
// has the rounding error of c m in its exponent, which is past 128 from 2^31 on).
// The weights enter as two bf16 terms (their sum holds 16 bits, and an output
// is then as exact as its own rounding), fp32 queries as three, which hold all
// of their 24 bits: lse is an fp32 result, and two terms left its scores' error
// at 2^-17 of them.  The matrix units idle most of the time here.
//
// Work split.  A unit is 128 tokens of one (sequence, key-value head, 16
// query heads), four waves with a tile each.  The units of the whole batch
// lie in one line, which the workgroups share out evenly, whatever the
// lengths: every workgroup works the line up from the device's lengths by
// itself.  The loads of a tile are in flight while the one before it is worked
// on, across the ends of rows too.  A row of units that ends up in several workgroups leaves fp32
// partial results (sum, maximum, unnormalised output) in the workspace, and
// join_kernel adds them in workgroup order.  Where the table has room for few
// units a row stays in one piece instead, and nothing is joined (see is_whole).
// Formed scores (kForm) are worked out between the products, on the lane's 8
// scores: cap tanh(scale q.k / cap) less the head's slope times the distance.
// They and the maximum are kept in units of the cap then.  Tokens before a
// sequence's first are none of its units'; those of the first group of 8 that
// come before it are masked as those behind the end are.
// fp32 queries' third term costs up to 4% (31 sequences of 4000 tokens, 32 heads
// of 256, e4m3 59.4 -> 61.8 us; of 128, bf16 52.6 -> 52.7).
#pragma once

#include "step_internal.h"

namespace bd {
namespace attend {

constexpr int kWaves = 4;
constexpr int kTile = 32;                  // tokens of a wave
constexpr int kUnit = kWaves * kTile;      // tokens of a unit
// A kernel's width: head_dim rounded up to 64, 96, 128, 192 or 256.  96 and 192
// against the next power of two, for which a load's lanes would idle: 31
// sequences of up to 1013 tokens, 32 heads, e4m3, 37.0 -> 30.8 us at 96 and 73.2
// -> 48.3 at 192 (fp32 queries).  Head sizes between go where their value loads
// are the better ones: 80 in bf16 to 128 (lanes of 8 columns, not 4 and 2; 64
// sequences of up to 2048, 32 heads, 148 there, 181 at 96), 144 to 176 in e4m3
// to 256 (of 16 columns, not 8 and 4; 176: 177 there, 206 at 192).
// e2m1 rows, which are a multiple of 32 wide, go to the next width, but for 96,
// which goes to 128 (lanes of 8 columns, not 4 and 2, whose loads of 2 bytes and 1
// took 293 us where 128 takes 128).
constexpr int width_of(int dim, int held) {
    return dim <= 64 ? 64 : (dim == 96 && held != BD_E2M1) || (dim < 96 && held == BD_E4M3) ? 96 : dim <= 128 ? 128 :
           dim == 192 || (dim < 192 && held != BD_E4M3) ? 192 : 256;
}
// Workgroups at most: what 256 CUs hold of them by their registers and LDS, so
// that all start at once.  Three per CU at width 64 (against two, 31
// sequences of 4000 tokens, 32 heads, e4m3: 135 -> 117 us), two at 128 (with
// 768 of them for 512 places, 64 of 8192 tokens in e4m3 173 -> 230 us) and at
// 192 (31 of up to 1013 tokens, 32 heads, e4m3: one 61.2, two 48.4).  At 256
// the registers of two spill but for e4m3 with bf16 queries (in bf16, 8 of 8192
// tokens, two would take 86 -> 107).  Of 4-bit codes with bf16 queries three up
// to 128, whose loads in flight are small (64 sequences of up to 16381 tokens, 64
// heads of 128 over 8, 132 -> 123 us, with a cap 141 -> 134; one of 131071 35.0 ->
// 35.4); shape_of says where they are launched.
constexpr int kCUs = 256;
constexpr int per_cu(int width, bool split_q, int held) {
    return width <= 64 || (width <= 128 && held == BD_E2M1 && !split_q) ? 3 : width <= 192 || (held != BD_BF16 && !split_q) ? 2 : 1;
}
// What a row costs beside its units, in units.  Without it the workgroups that
// get many short rows come last: 64 sequences of up to 16381 tokens in e4m3
// 187 -> 178 us, 31 of up to 1013 with 32 key-value heads 27.7 -> 22.7 (16 of
// up to 4099 in bf16 28.9 -> 30.0).
constexpr int kRowCost = 2;
constexpr float kLazy = 10.0f;             // log2: how large a weight may be before the maximum moves
constexpr float kNegInf = -__builtin_inff();
// Times the least fp32 number -infinity (a score behind the end) stays what it is,
// times 0 it would not; and no difference of scores times it is worth 2^-20.
constexpr float kLeastC = 0x1p-149f;

struct Shape {
    int32_t heads, dim, page_size, pg8, magic;  // pg8: groups of 8 tokens in a page
    int32_t group, tiles;                       // query heads per kv head, and tiles of 16 of them
    int32_t rows;                               // rows of units per sequence: heads * tiles
    int32_t capacity, groups;                   // tokens a table row holds; workgroups launched
    int32_t crosses, by_row;                    // entries of the workspace's table
    int32_t whole;                              // rows stay in one piece, see is_whole
    int32_t ordered;                            // of them, a workgroup each, the longest first
};

struct Args {
    AttendArgs a;
    Shape s;
    uint32_t pages;                         // of the cache
    uint32_t page16, head16, token16;       // its strides in units of 16 bytes
    uint32_t page_scales, head_scales;      // scale bytes of a page, of a head of it
    // what the maximum's units take to be exponents of 2, no smaller than kLeastC, and to be scores
    float c, unit;
    float times;                            // what a product takes to be a formed score
    uint32_t flip;                          // the queries' sign bits where scale is negative
};

// The logarithm of a row's sum from its maximum (of the scores, which have the
// sign of scale in them) and its sum of weights.
__device__ __forceinline__ float lse_of(const Args& p, float m, float l) {
    return __builtin_fmaf(m, p.unit, __builtin_amdgcn_logf(l) * 0.69314718055994531f);
}

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Units of one row of a sequence: at least one, so that an empty sequence's
// outputs are written too; one where the length is out of range.
__device__ __forceinline__ int units_of(int len, int capacity) {
    return len <= kUnit || len > capacity ? 1 : (len + kUnit - 1) / kUnit;
}

// A sequence's length and its first token attended to, 0 .. length - 1; a
// sequence of no tokens attended to has length 0.
struct Seq {
    int len, first;
    __device__ __forceinline__ int base() const { return first & ~7; }  // the first of its units' tokens
    __device__ __forceinline__ int units(int capacity) const { return units_of(len - base(), capacity); }
};
template <bool kForm>
__device__ __forceinline__ Seq seq_of(const Args& p, int b) {
    Seq s{p.a.lengths[b], 0};
    if (kForm && p.a.first) {
        s.first = p.a.first[b];
        if (s.first < 0 || s.len > p.s.capacity) s.first = 0;
        if (s.first >= s.len && s.len <= p.s.capacity) s = Seq{0, 0};
    }
    return s;
}

// The batch's line of places, worked out by each wave: a row has kRowCost of
// them for its start and end (queries, sums over the waves, outputs) and one
// for each of its units.  Lane l sums the sequences [l n, l n + n).
__device__ __forceinline__ Seq uni_seq(Seq s) { return Seq{uni(s.len), uni(s.first)}; }
template <bool kForm>
struct Line {
    int n, first, total;  // per lane: sequences, places before its own; places of the batch
    Seq seq;              // per lane: its last sequence
    __device__ __forceinline__ void scan(const Args& p) {
        const int lane = threadIdx.x & 63;
        n = (p.a.B + 63) / 64;
        int sum = 0;
        const int b0 = lane * n;
        seq = Seq{0, 0};
        for (int i = 0; i < n; ++i)
            if (b0 + i < p.a.B) {
                seq = seq_of<kForm>(p, b0 + i);
                sum += kRowCost + seq.units(p.s.capacity);
            }
        sum *= p.s.rows;
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        first = inc - sum;
        total = uni(__shfl(inc, 63, 64));
    }
    // The sequence that holds place u, its first place and its tokens.
    __device__ __forceinline__ int holder_of(const Args& p, int u, int* start, Seq* held) const {
        const int lane = threadIdx.x & 63;
        // the last lane that has sequences and starts at or before u
        const uint64_t at = __ballot(lane * n < p.a.B && first <= u);
        const int l = 63 - __clzll(at);
        int s = uni(__shfl(first, l, 64));
        if (n == 1) {
            *start = s;
            *held = Seq{uni(__shfl(seq.len, l, 64)), kForm ? uni(__shfl(seq.first, l, 64)) : 0};
            return uni(l);
        }
        int b = l * n;
        for (;;) {
            *held = uni_seq(seq_of<kForm>(p, b));
            const int span = (kRowCost + held->units(p.s.capacity)) * p.s.rows;
            if (u < s + span || b + 1 >= p.a.B) break;
            s += span;
            ++b;
        }
        *start = uni(s);
        return uni(b);
    }
};

// Of at most kSorted sequences the one that has `rank` before it when they are
// sorted by falling units, then by index.
constexpr int kSorted = 256;
template <bool kForm>
__device__ __forceinline__ int sequence_of_rank(const Args& p, int rank, Seq* held) {
    const int lane = threadIdx.x & 63;
    Seq seq[kSorted / 64];
    int units[kSorted / 64];
#pragma unroll
    for (int i = 0; i < kSorted / 64; ++i) {
        const bool own = i * 64 + lane < p.a.B;
        seq[i] = own ? seq_of<kForm>(p, i * 64 + lane) : Seq{0, 0};
        units[i] = own ? seq[i].units(p.s.capacity) : 0;
    }
    for (int u = (p.s.capacity + kUnit - 1) / kUnit; u >= 1; --u) {
#pragma unroll
        for (int i = 0; i < kSorted / 64; ++i) {
            if (i * 64 >= p.a.B) break;
            const uint64_t of = __ballot(units[i] == u);
            const int n = __popcll(of);
            if (rank < n) {
                const int before =
                    __builtin_amdgcn_mbcnt_hi((uint32_t)(of >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)of, 0));
                const int l = uni(__ffsll((unsigned long long)__ballot(before == rank && units[i] == u)) - 1);
                held->len = __builtin_amdgcn_readlane(seq[i].len, l);
                held->first = kForm ? __builtin_amdgcn_readlane(seq[i].first, l) : 0;
                return i * 64 + l;
            }
            rank -= n;
        }
    }
    *held = Seq{0, 0};
    return 0;  // not reached: the ranks are those of the sequences
}

// Workgroup w of W takes the places [start(w), start(w + 1)).  A row's units
// before place u are those of its places before u, less kRowCost: what is cut
// within a row's cost starts with the row's first unit.
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
// places (the first row it works on and the last one) of 16 (maximum, sum) and a
// row's heads' unnormalised outputs.
//
// Cross: a row of units that starts in one workgroup and goes on in the next
// ones.  The table has an entry per row of the batch where these are fewer
// than the workgroups, else one per workgroup (in which at most one such row
// starts); each is written in every call.
struct Cross {
    int32_t id;     // b * rows + row
    int32_t first;  // the workgroup it starts in, times 2, plus its place there; -1: all of it is in one workgroup
    int32_t last;   // the workgroup it ends in
    int32_t pad;
};
// Numbers of a place, whose heads are 16, or past 64 columns no more than a row's
// (see shape_of).
__host__ __device__ __forceinline__ constexpr int heads_of_place(int dim, int group) { return dim <= 64 || group >= 16 ? 16 : group; }
__host__ __device__ __forceinline__ constexpr int numbers_of_place(int dim, int group) { return 32 + heads_of_place(dim, group) * dim; }
__device__ __forceinline__ float* place(const Args& p, int w, int which) {
    return p.a.part + (int64_t)p.s.crosses * 4 + ((int64_t)w * 2 + which) * numbers_of_place(p.s.dim, p.s.group);
}

// Page lookups: token group g8 (8 tokens, which no page boundary cuts) of a
// sequence lies in page table[g8 / pg8], at group g8 % pg8 of it.
struct Group {
    int page, in_page;
};
__device__ __forceinline__ Group look_up(const Shape& s, const int32_t* table, int g8) {
    // exact: g8 < 2^21, pg8 <= 2^9
    const uint32_t idx = __umulhi((uint32_t)g8, (uint32_t)s.magic) + (s.pg8 == 1 ? g8 : 0);
    return Group{table[idx], g8 - (int)__umul24(idx, (uint32_t)s.pg8)};
}
struct Where {
    uint64_t at;  // byte of the group's first token in the cache's arrays
    uint64_t sc;  // its scale byte
    bool bad;
};
__device__ __forceinline__ Where locate(const Args& p, Group x, int head) {
    Where w;
    w.bad = (uint32_t)x.page >= p.pages;
    const uint32_t page = w.bad ? 0u : (uint32_t)x.page, at = (uint32_t)x.in_page * 8;
    w.at = ((uint64_t)page * p.page16 + ((uint64_t)at * p.token16 + (uint64_t)(uint32_t)head * p.head16)) * 16;
    w.sc = (uint64_t)page * p.page_scales + ((uint32_t)head * p.head_scales + at);
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
    if constexpr (N == 0) {
    } else if constexpr (N == 1) {
        r.d[0] = *static_cast<const uint32_t*>(p);  // rows of half a cache line, whose other half comes next
    } else if constexpr (N == 2) {
        typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
        const u32x2_t v = __builtin_nontemporal_load(static_cast<const u32x2_t*>(p));
        r.d[0] = v.x, r.d[1] = v.y;
    } else if constexpr (N % 4) {
#pragma unroll
        for (int i = 0; i < N; ++i) r.d[i] = __builtin_nontemporal_load(static_cast<const uint32_t*>(p) + i);
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

// Two e2m1 codes, byte i of a lane's dwords, as a bf16 pair.
__device__ __forceinline__ uint32_t e2m1_pair(uint32_t w, float scale, int byte) {
    switch (byte) {
        case 0: return e2m1x2_to_bf16<0>(w, scale);
        case 1: return e2m1x2_to_bf16<1>(w, scale);
        case 2: return e2m1x2_to_bf16<2>(w, scale);
        default: return e2m1x2_to_bf16<3>(w, scale);
    }
}

__device__ __forceinline__ void flip(uint4& v, uint32_t mask) { v.x ^= mask, v.y ^= mask, v.z ^= mask, v.w ^= mask; }

// The scores of 8 consecutive tokens from their products, `far` the first one's
// distance to the new token.
__device__ __forceinline__ void form_scores(const Args& p, float* sc, float times, float slope, int far) {
    if (p.a.cap > 0.0f) {
        cap_scores<8>(sc, times);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] *= times;
    }
    if (p.a.slopes) {
#pragma unroll
        for (int j = 0; j < 8; ++j) sc[j] = __builtin_fmaf(-slope, (float)(far - j), sc[j]);
    }
}

// kDC: the width, see width_of.  kFull: head_dim is kDC.  kHeld: the cache's type.
// kSplitQ: fp32 queries as three bf16 terms.  kForm: formed scores.
template <int kDC, bool kFull, int kHeld, bool kSplitQ, bool kForm>
__global__ __launch_bounds__(kWaves * 64, per_cu(kDC, kSplitQ, kHeld)) void attend_kernel(const Args p) {
    constexpr bool kE4m3 = kHeld == BD_E4M3, kE2m1 = kHeld == BD_E2M1;
    constexpr int NS = kDC / 32;              // k-steps of a score product
    constexpr int kBits = kE2m1 ? 4 : kE4m3 ? 8 : 16;  // of a held value
    // Loads of a key row per lane, 16 bytes each, but the last one of e4m3 8 where
    // the k-steps are odd (one k-step of codes), and the last ones of e2m1 for two
    // k-steps or one, 8 and 4 bytes.  k_steps, k_first: of load s.
    constexpr int KL = kE2m1 ? NS / 4 + (NS % 4 + 1) / 2 : (NS * kBits / 8 + 1) / 2;
    constexpr bool kOdd = kE4m3 && NS % 2;
    const auto k_steps = [](int s) { return s < NS / 4 ? 4 : s == NS / 4 && NS % 4 >= 2 ? 2 : 1; };
    const auto k_first = [](int s) { return s <= NS / 4 ? 4 * s : NS / 4 * 4 + 2; };
    // Value columns of a lane: DV1 neighbouring ones of the first 16 DV1, and
    // where those are not all, DV2 neighbouring ones of the rest (at 96 and 192,
    // where a lane's share of all columns is no load's size, or ends past head_dim).
    constexpr int DV = kDC / 16, DV1 = DV % 3 == 0 && (!kFull || DV * kBits % 32) ? DV / 3 * 2 : DV, DV2 = DV - DV1;
    constexpr int kMin = kDC == 64 ? 0 : kDC <= 128 ? 64 : 128;  // head_dim is more than that
    constexpr int VD = (DV * kBits + 31) / 32;  // dwords of a value row per lane
    constexpr int VB1 = DV1 * kBits / 8, VB2 = DV2 * kBits / 8;
    constexpr int kPad = kDC + 4;
    // Two of each, used in turn by the rows: one barrier a row.  One where a CU
    // then holds a workgroup more: past head_dim 128 two instead of one (at 256,
    // and for fp32 queries, with the queries in LDS instead of registers), at 128
    // three instead of two.
    constexpr bool kOneTurn = kDC > 64 && per_cu(kDC, kSplitQ, kHeld) > (kDC > 128 ? 1 : 2);
    constexpr bool kTight = kOneTurn && kDC > 128 && (kDC == 256 || kSplitQ);
    constexpr int QT = kSplitQ ? 3 : 1;
    constexpr int kTurns = kOneTurn ? 1 : 2;
    __shared__ float so[kTurns][kWaves][16][kPad];
    __shared__ float sm[kTurns][kWaves][16], sl[kTurns][kWaves][16];
    __shared__ uint4 sq[kTight ? QT : 1][kTight ? NS : 1][64];
    // What a masked token's values are is settled after the weights where that
    // lets the values come later: e2m1 without formed scores 136 -> 129 us, with
    // a cap 149 -> 152 (64 sequences of up to 16381 tokens, 64 heads of 128 over 8).
    constexpr bool kLate = kE2m1 && !kForm;
    // Whether page numbers are sent before the keys of the tile before and scale
    // bytes made scales where they are used, see below.  Without formed scores only
    // where that gives something.  Not in e4m3 from 128 columns on (31 sequences of up
    // to 1013 tokens, 32 heads of 128 / 192 / 256, 37.1 -> 36.0 / 50.5 -> 48.7 / 64.7
    // -> 62.0 us; 64 of up to 16381, 64 heads over 8, at 192 294 -> 290), but with fp32
    // queries of 256 (there 80.2 -> 74.5).  In bf16 at 160 to 192 and 256 (32 of up to
    // 8192, 32 heads over 8, 168 -> 165.5 and 228 -> 216), not below or between (16 of
    // up to 300, 64 heads of 64 6.75 -> 6.86; 4 of up to 37, of 224, 8.4 -> 8.8).
    constexpr bool kPagesFirst = kE2m1 || kForm || (kE4m3 ? kDC < 128 || (kDC == 256 && kSplitQ)
                                                          : kDC == 192 || (kDC == 256 && kFull));
    // Whether a tile's next loads are sent in any case, see below.  Not where that
    // is more than it gives: in bf16 without formed scores (at 256 32 of up to 8192
    // 216 -> 220, 16 of up to 300 18.6 -> 19.4, with formed ones up to 128, where no
    // scales are waited for) and in e4m3 at 64 without them (31 of up to 1013, 32
    // heads, 20.9 -> 21.9; with a bias by distance 16 of up to 8191 67.7 -> 65.2; at
    // 96 64 of up to 16381 160 -> 157, at 256 with fp32 queries 392 -> 360).
    constexpr bool kAlways = kPagesFirst && (kE2m1 || (kForm && kDC > 128) || (kE4m3 && (kForm || kDC > 64)));
    constexpr int NR = kTight ? (NS + kWaves - 1) / kWaves : NS;  // k-steps whose queries a wave loads

    const int lane = threadIdx.x & 63, wave = uni(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    // rows in one piece: a row is one place of the line, which needs no lengths
    const bool whole = p.s.whole;
    const int cost = whole ? 0 : kRowCost;
    Line<kForm> line;
    if (!whole) line.scan(p);
    const Cut cut(whole ? p.a.B * p.s.rows : line.total, p.s.groups);
    const int w = blockIdx.x;
    Cross* crosses = reinterpret_cast<Cross*>(p.a.part);
    const bool by_row = p.s.by_row;
    if (!by_row && crosses && threadIdx.x == 0) crosses[w].first = -1;
    if (w >= cut.W) return;
    const int u = cut.start(w);
    const int end = cut.start(w + 1);
    int at, b0;  // the current row's first place; the first sequence
    Seq seq0;
    if (whole) {
        b0 = u / p.s.rows;
        at = b0 * p.s.rows;
        if (p.s.ordered) {
            b0 = sequence_of_rank<kForm>(p, b0, &seq0);
        } else {
            seq0 = uni_seq(seq_of<kForm>(p, b0));
        }
    } else {
        b0 = line.holder_of(p, u, &at, &seq0);
    }

    // The part of a row of units that this workgroup works on.
    struct Piece {
        int b, row, unit, n, un;     // sequence, its row, first unit, units here, units of the row
        int len, tokens, t0, stop;   // length as given and as used; this wave's first tile, its tokens' end
        int first;                   // the first token attended to
        int head, q0, nq;            // key-value head; first query head of its group, and how many
    };
    const auto piece_at = [&](int b, Seq seq, int row, int unit, int row_at) {
        Piece x;
        x.b = b, x.row = row, x.unit = unit, x.len = seq.len, x.first = kForm ? seq.first : 0;
        x.un = seq.units(p.s.capacity);
        const int base = kForm ? seq.base() : 0;
        const int upto = end - row_at - kRowCost;  // of its units, as far as this workgroup goes
        x.n = (whole || upto >= x.un ? x.un : upto) - unit;
        x.tokens = x.len > p.s.capacity || x.len < 0 ? 0 : x.len;
        x.t0 = base + unit * kUnit + wave * kTile;
        const int end_of = base + (unit + x.n) * kUnit;
        x.stop = x.tokens < end_of ? x.tokens : end_of;
        x.head = row / p.s.tiles;
        x.q0 = (row - x.head * p.s.tiles) * 16;
        x.nq = p.s.group - x.q0 < 16 ? p.s.group - x.q0 : 16;
        return x;
    };
    const int span0 = whole ? 1 : kRowCost + seq0.units(p.s.capacity), row0 = (u - at) / span0;
    at += row0 * span0;
    if (at + cost >= end) return;  // no unit of its own
    const int into = u - at - cost;
    Piece now = piece_at(b0, seq0, row0, into > 0 ? into : 0, at);
    bool first_piece = true;

    // A tile's loads, in flight while the tile before it is worked on: the keys
    // as soon as the scores are done with the registers, the values after the
    // sums, the page numbers just before the keys of the tile before, so that none is
    // waited for by way of another that was sent later (kPagesFirst; else after the
    // values).  Behind a piece's last tile page 0 is loaded, whose lines all waves
    // share (kAlways): without a branch the compiler knows what is on its way at a
    // tile's start, and does not wait for all of it.
    // (64 sequences of up to 16381 tokens, 64 heads of 128 over 8, e2m1: 155 ->
    // 129 us; 16 of up to 8191, 32 heads of 64, e4m3, a bias by distance: 72 -> 63.)
    // A row's first tile and its queries are loaded while the row before it is
    // summed up.
    Dwords<4> kk[2][KL];  // of the odd one, two
    Dwords<VD> vv[8];
    constexpr int KG = kE2m1 ? KL : 1, VG = kE2m1 && DV2 > 0 ? 2 : 1;  // scales of a lane's part of a row
    uint32_t ks[2][KG];
    uint2 vs[VG];
    float slope = 0.0f;  // of the lane's head
    Raw8<kSplitQ> raw[NR];
    bool bad = false;
    const auto group_of = [&](const Piece& x, int t, int add) {
        const int g8 = (t >> 3) + add, last = (x.tokens - 1) >> 3;
        return g8 < last ? g8 : last;  // (a piece's first tile starts in its first group)
    };
    // The one after x, in the same sequence or the next.
    const auto piece_after = [&](const Piece& x, int row_at) {
        const bool over = x.row + 1 == p.s.rows;
        const int b = x.b + over;
        return piece_at(b, over ? uni_seq(seq_of<kForm>(p, b)) : Seq{x.len, x.first}, over ? 0 : x.row + 1, 0, row_at);
    };
    // where the lane's key rows and value rows are
    struct Groups {
        Group k, v;
    };
    const auto load_pages = [&](const Piece& x, int t) {
        const int32_t* table = p.a.table + x.b * p.a.table_stride;
        return Groups{look_up(p.s, table, group_of(x, t, i16 >> 2)), look_up(p.s, table, group_of(x, t, g))};
    };
    const uint64_t token_bytes = (uint64_t)p.token16 * 16;
    const auto load_keys = [&](const Where& wh) {
        bad |= wh.bad;
        // one address, stepped by uniform strides, so that no per-row address
        // stays in registers
        uint64_t at = opaque(wh.at + (uint64_t)(i16 & 3) * token_bytes + (kE2m1 ? 0 : g * 16));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int s = 0; s < KL; ++s) {
                clear(kk[h][s]);
                if constexpr (kE2m1) {
                    const int steps = k_steps(s), d = k_first(s) * 32 + g * steps * 8;
                    const char* k = static_cast<const char*>(p.a.kv.k) + at + k_first(s) * 16 + g * (steps * 4);
                    if (kFull || k_first(s) * 32 + 32 * steps <= kMin || d < p.s.dim) {
                        if (steps == 4) {
                            kk[h][s] = load_dwords<4>(k);
                        } else if (steps == 2) {
                            const Dwords<2> r = load_dwords<2>(k);
                            kk[h][s].d[0] = r.d[0], kk[h][s].d[1] = r.d[1];
                        } else {
                            kk[h][s].d[0] = load_dwords<1>(k).d[0];
                        }
                    }
                    // the lane's columns of a load lie in one group
                    const int group = kFull || d < p.s.dim ? d / kGroup4 : 0;
                    ks[h][s] = p.a.kv.k_scales[wh.sc + (uint32_t)group * (uint32_t)p.s.page_size + (i16 & 3) + 4 * h];
                    continue;
                }
                const char* k = static_cast<const char*>(p.a.kv.k) + at + s * 64;
                if (kOdd && s == KL - 1) {
                    if (kFull || s * 64 + 32 <= kMin || s * 64 + g * 8 < p.s.dim) {
                        const Dwords<2> r = load_dwords<2>(k - g * 8);
                        kk[h][s].d[0] = r.d[0], kk[h][s].d[1] = r.d[1];
                    }
                } else if (kFull || (s * 64 + 64) * 8 / kBits <= kMin || (s * 64 + g * 16) * 8 / kBits < p.s.dim) {
                    kk[h][s] = load_dwords<4>(k);
                }
            }
            at += 4 * token_bytes;
            if (kE4m3) {
                const uint32_t byte = p.a.kv.k_scales[wh.sc + (i16 & 3) + 4 * h];
                ks[h][0] = kPagesFirst ? byte : __float_as_uint(scale_of(byte));
            }
        }
    };
    const auto load_values = [&](const Where& wh) {
        bad |= wh.bad;
        // lanes behind head_dim hold some other columns, which are not used
        uint64_t at = opaque(wh.at + (kFull || i16 * DV1 < p.s.dim ? i16 * VB1 : 0));
        const uint32_t rest = DV2 == 0 ? 0 : kFull || 16 * DV1 + i16 * DV2 < p.s.dim ? 16 * VB1 + i16 * VB2 : 0;
        uint64_t at2 = opaque(wh.at + rest);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const char* v = static_cast<const char*>(p.a.kv.v) + at;
            if constexpr (VB1 == 2) {
                vv[j].d[0] = *reinterpret_cast<const uint16_t*>(v);
            } else {
                const Dwords<VB1 / 4> r = load_dwords<VB1 / 4>(v);
#pragma unroll
                for (int i = 0; i < VB1 / 4; ++i) vv[j].d[i] = r.d[i];
            }
            at += token_bytes;
            const char* v2 = static_cast<const char*>(p.a.kv.v) + at2;
            if constexpr (VB2 == 1) {
                vv[j].d[0] |= (uint32_t)*reinterpret_cast<const uint8_t*>(v2) << 16;
            } else if constexpr (VB2 == 2) {
                vv[j].d[VD - 1] = *reinterpret_cast<const uint16_t*>(v2);
            } else {
                const Dwords<VB2 / 4> r2 = load_dwords<VB2 / 4>(v2);
#pragma unroll
                for (int i = 0; i < VB2 / 4; ++i) vv[j].d[VB1 / 4 + i] = r2.d[i];
            }
            if constexpr (DV2 > 0) at2 += token_bytes;
        }
        if (kE4m3) vs[0] = *reinterpret_cast<const uint2*>(p.a.kv.v_scales + wh.sc);
        if constexpr (kE2m1) {
            const uint32_t rows = (uint32_t)p.s.page_size;
            const int c0 = kFull || i16 * DV1 < p.s.dim ? i16 * DV1 : 0;
            vs[0] = *reinterpret_cast<const uint2*>(p.a.kv.v_scales + wh.sc + (uint32_t)(c0 / kGroup4) * rows);
            if constexpr (VG == 2) {
                const int c1 = kFull || 16 * DV1 + i16 * DV2 < p.s.dim ? 16 * DV1 + i16 * DV2 : 0;
                vs[VG - 1] = *reinterpret_cast<const uint2*>(p.a.kv.v_scales + wh.sc + (uint32_t)(c1 / kGroup4) * rows);
            }
        }
    };
    // queries: B operand, column i16, k = the head's values in the order in
    // which the key loads bring them
    const auto load_queries = [&](const Piece& x) {
        const int64_t at = x.b * p.a.qs.token + (x.head * p.s.group + x.q0 + i16) * p.a.qs.head;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int s = kTight ? i * kWaves + wave : i;
            int d = kE4m3 && !(kOdd && s == NS - 1) ? (s >> 1) * 64 + g * 16 + (s & 1) * 8 : s * 32 + g * 8;
            if (kE2m1) {
                const int l = s < NS / 4 * 4 ? s / 4 : s < NS / 4 * 4 + k_steps(NS / 4) ? NS / 4 : NS / 4 + 1;
                d = k_first(l) * 32 + (g * k_steps(l) + s - k_first(l)) * 8;
            }
            raw[i].zero();
            if (s < NS && i16 < x.nq && (kFull || d < p.s.dim)) raw[i].load(p.a.q, at + d);
        }
        if (kForm && p.a.slopes) slope = i16 < x.nq ? p.a.slopes[x.head * p.s.group + x.q0 + i16] : 0.0f;
    };

    const auto drop = [&]() {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int s = 0; s < KL; ++s) clear(kk[h][s]);
#pragma unroll
        for (int j = 0; j < 8; ++j) clear(vv[j]);
#pragma unroll
        for (int i = 0; i < KG; ++i) ks[0][i] = ks[1][i] = 0;
#pragma unroll
        for (int i = 0; i < VG; ++i) vs[i] = make_uint2(0, 0);
    };

    Groups pages{};  // of the tile after the one in flight
    // The page numbers of the tile at t and the keys of the one before it, or of
    // page 0; its values are at what comes back.
    const auto load_next = [&](const Piece& x, int t, bool more) {
        const Where k = locate(p, more ? pages.k : Group{0, 0}, x.head);
        if constexpr (!kPagesFirst) {
            load_keys(k);
            return Where{};
        } else {
            const Where v = locate(p, more ? pages.v : Group{0, 0}, x.head);
            __builtin_amdgcn_sched_barrier(0);  // no copies of numbers that are on their way
            pages = load_pages(x, t);           // past the end: the last group's page
            __builtin_amdgcn_sched_barrier(0);
            load_keys(k);
            __builtin_amdgcn_sched_barrier(0);
            return v;
        }
    };
    // That tile's values, and where they come first the page numbers of the next.
    const auto load_rest = [&](const Piece& x, int t, const Where& v) {
        if constexpr (!kPagesFirst) {
            load_values(locate(p, pages.v, x.head));
            pages = load_pages(x, t);
        } else {
            load_values(v);
        }
    };
    drop();
    load_queries(now);
    if (now.t0 < now.stop) {
        pages = load_pages(now, now.t0);
        load_rest(now, now.t0 + kUnit, load_next(now, now.t0 + kUnit, true));
    }

    for (int turn = 0;; turn ^= kTurns - 1) {
        const int t0 = now.t0, stop = now.stop, nq = now.nq, tokens = now.tokens, len = now.len, first = now.first;
        // what comes next, and its first page numbers
        const int next_at = at + (whole ? 1 : kRowCost + now.un);
        const bool last = next_at + cost >= end;
        Groups next_pages{};
        if (!last) {
            const Piece next = piece_after(now, next_at);
            if (next.t0 < next.stop) next_pages = load_pages(next, next.t0);
        }

        uint4 qt[QT][NR];  // the terms, the largest first
#pragma unroll
        for (int s = 0; s < NR; ++s) {
            if constexpr (kSplitQ) {
                float f[8], back[8];
                raw[s].widen(f);
#pragma unroll
                for (int k = 0; k < QT; ++k) {
                    qt[k][s] = narrow_bf16x8(f);
                    widen_bf16x8(qt[k][s], back);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] -= back[j];
                }
            } else {
                qt[0][s] = raw[s].a;
            }
            raw[s].zero();  // not kept through the tiles
#pragma unroll
            for (int k = 0; k < QT; ++k) {
                flip(qt[k][s], p.flip);
                if (kTight && s * kWaves + wave < NS) sq[k][s * kWaves + wave][lane] = qt[k][s];
            }
        }
        if constexpr (kTight) __syncthreads();

        f32x4_t acc[DV];
        float m, mm, l;  // mm: m, or 0 while m is -infinity
        float c = p.c, times = kForm ? p.times : 1.0f;
        const float bias = kForm ? slope_in(slope, p.unit) : 0.0f;
        int pass = 0;  // 1: again, see below
        bool lost = false;

    again:
#pragma unroll
        for (int j = 0; j < DV; ++j) acc[j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        m = kNegInf, mm = 0.0f, l = 0.0f;
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
                        const float scale = kPagesFirst ? scale_of(ks[h][0]) : __uint_as_float(ks[h][0]);
                        kb = make_uint4(e4m3x2_to_bf16<false>(c0, scale), e4m3x2_to_bf16<true>(c0, scale),
                                        e4m3x2_to_bf16<false>(c1, scale), e4m3x2_to_bf16<true>(c1, scale));
                    } else if constexpr (kE2m1) {
                        const int l = s < NS / 4 * 4 ? s / 4 : s < NS / 4 * 4 + k_steps(NS / 4) ? NS / 4 : NS / 4 + 1;
                        kb = e2m1x8_to_bf16(kk[h][l].d[s - k_first(l)], scale_of(ks[h][l]));
                    } else {
                        const Dwords<4>& r = kk[h][s];
                        kb = make_uint4(r.d[0], r.d[1], r.d[2], r.d[3]);
                    }
#pragma unroll
                    for (int k = QT - 1; k >= 0; --k) {
                        uint4 qk;
                        if constexpr (kTight)
                            qk = sq[lost ? 0 : k][s][lane];
                        else
                            qk = qt[k][s];
                        x = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(kb), as_bf16x8(qk), x, 0, 0, 0);
                    }
                    if (kTight && kSplitQ) __builtin_amdgcn_sched_barrier(0);  // or all terms wait in registers
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[4 * h + r] = x[r];
            }
            Where values_at{};
            if (kAlways || more) values_at = load_next(now, t + 2 * kUnit, more);
            if constexpr (kForm) form_scores(p, sc, times, bias, len - 1 - (t + 8 * g));
            const bool tail = t + kTile > tokens || (kForm && t < first);
            const auto clear_value = [&](int j, bool out) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < VD; ++i) vv[j].d[i] = out ? 0u : vv[j].d[i];
                if constexpr (kHeld != BD_BF16) {  // any byte may stand there: 2^0
#pragma unroll
                    for (int i = 0; i < VG; ++i) {
                        uint32_t& sw = j < 4 ? vs[i].x : vs[i].y;
                        const uint32_t field = 0xffu << (8 * (j & 3));
                        sw = out ? (sw & ~field) | (127u << (8 * (j & 3))) : sw;
                    }
                }
            };
            if (tail) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const bool out = t + 8 * g + j >= tokens || (kForm && t + 8 * g + j < first);
                    sc[j] = out ? kNegInf : sc[j];
                    if constexpr (!kLate) clear_value(j, out);
                }
            }

            float mx = sc[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) mx = fmaxf(mx, sc[j]);
            if (__ballot((mx - m) * c > kLazy)) {
                mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
                mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
                const float up = fmaxf(m, mx);
                const float to = up == kNegInf ? 0.0f : up;
                const float f = __builtin_amdgcn_exp2f((m - to) * c);
                m = up;
                mm = to;
                l *= f;
#pragma unroll
                for (int j = 0; j < DV; ++j) acc[j] *= f;
            }
            float pr[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                pr[j] = __builtin_amdgcn_exp2f((sc[j] - mm) * c);
                l += pr[j];
            }
            const uint4 ph = narrow_bf16x8(pr);
            float back[8];
            widen_bf16x8(ph, back);
#pragma unroll
            for (int j = 0; j < 8; ++j) back[j] = pr[j] - back[j];
            uint4 pl = narrow_bf16x8(back);
            if (pass) pl = ph;

            if (kLate && tail) {
#pragma unroll
                for (int j = 0; j < 8; ++j) clear_value(j, t + 8 * g + j >= tokens);
            }

            // value rows as bf16 pairs of columns, then pairs of tokens
            float vscale[VG][8];
            if constexpr (kHeld != BD_BF16) {
#pragma unroll
                for (int i = 0; i < VG; ++i)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        vscale[i][j] = scale_of(((j < 4 ? vs[i].x : vs[i].y) >> (8 * (j & 3))) & 0xff);
            }
#pragma unroll
            for (int i = 0; i < DV / 2; ++i) {
                uint32_t vb[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if constexpr (kE4m3)
                        vb[j] = i & 1 ? e4m3x2_to_bf16<true>(vv[j].d[i / 2], vscale[0][j])
                                      : e4m3x2_to_bf16<false>(vv[j].d[i / 2], vscale[0][j]);
                    else if constexpr (kE2m1)
                        vb[j] = e2m1_pair(vv[j].d[i / 4], vscale[i < DV1 / 2 ? 0 : VG - 1][j], i & 3);
                    else
                        vb[j] = vv[j].d[i];
                }
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    uint32_t va[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        va[k] = __builtin_amdgcn_perm(vb[2 * k + 1], vb[2 * k], o ? 0x07060302u : 0x05040100u);
                    const bf16x8_t av = as_bf16x8(make_uint4(va[0], va[1], va[2], va[3]));
                    f32x4_t& a = acc[2 * i + o];
                    a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, as_bf16x8(pl), a, 0, 0, 0);
                    a = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, as_bf16x8(ph), a, 0, 0, 0);
                }
                if (kTight) __builtin_amdgcn_sched_barrier(0);  // or the pairs of all columns wait in registers
            }
            if (kAlways || more) load_rest(now, t + 2 * kUnit, values_at);
        }

        // Further terms break on infinities: they are of either sign or zero,
        // and infinity minus itself or times zero is NaN.  So where a sum is
        // not finite the wave goes over its tokens again with one term, taken
        // as often as there are terms and divided by their number, and takes
        // what was lost from there.  The queries' further terms only go where
        // the scores broke.
        if (!pass) {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < DV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) z = __builtin_fmaf(acc[j][r], 0.0f, z);
            if (__ballot(i16 < nq && (z != 0.0f || l != l))) {
                lost = kSplitQ && __ballot(i16 < nq && l != l);
                float* keep = &so[turn][wave][0][0] + lane;
#pragma unroll
                for (int j = 0; j < DV; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) keep[(4 * j + r) * 64] = acc[j][r];
                if (lost) {
#pragma unroll
                    for (int s = 0; s < NR; ++s)
#pragma unroll
                        for (int k = 1; k < QT; ++k) qt[k][s] = qt[0][s];
                    if (kForm)
                        times *= 1.0f / QT;
                    else
                        c = fmaxf(c * (1.0f / QT), kLeastC);
                }
                pass = 1;
                pages = load_pages(now, t0);
                load_rest(now, t0 + kUnit, load_next(now, t0 + kUnit, true));
                goto again;
            }
        } else {
            const float* keep = &so[turn][wave][0][0] + lane;
#pragma unroll
            for (int j = 0; j < DV; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float x = keep[(4 * j + r) * 64];
                    acc[j][r] = !lost && x * 0.0f == 0.0f ? x : acc[j][r] * 0.5f;
                }
            if (lost && !kForm) m *= 1.0f / QT;  // of scores taken that often
        }

        // worked out again, so that it takes no registers through the tiles
        Piece from = now;
        asm("" : "+s"(from.row), "+s"(from.b));
        const Piece next = last ? now : piece_after(from, next_at);
        const bool was_bad = __ballot(bad) != 0 || now.len > p.s.capacity;
        bad = false;
        if (!last) load_queries(next);
        if (!last && next.t0 < next.stop) {
            pages = next_pages;
            load_rest(next, next.t0 + kUnit, load_next(next, next.t0 + kUnit, true));
        } else {  // nothing is kept in these registers from here
            drop();
        }

        // the wave's result, then the workgroup's: heads i16, values
        // (4 g + r) DV1 + j of acc[j][r], 16 DV1 + (4 g + r) DV2 + j of acc[DV1 + j][r]
        l += __shfl_xor(l, 16, 64);
        l += __shfl_xor(l, 32, 64);
        if (was_bad) l = __builtin_nanf("");
        if (lane < 16) sm[turn][wave][i16] = m, sl[turn][wave][i16] = l;
        if (i16 < nq) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = 0; j < DV1; j += DV1 % 4 ? 2 : 4) {
                    float* o = &so[turn][wave][i16][(4 * g + r) * DV1 + j];
                    if constexpr (DV1 % 4)
                        *reinterpret_cast<float2*>(o) = make_float2(acc[j][r], acc[j + 1][r]);
                    else
                        *reinterpret_cast<float4*>(o) =
                            make_float4(acc[j][r], acc[j + 1][r], acc[j + 2][r], acc[j + 3][r]);
                }
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int j = DV1; j < DV; j += 2)
                    *reinterpret_cast<float2*>(&so[turn][wave][i16][16 * DV1 + (4 * g + r) * DV2 + j - DV1]) =
                        make_float2(acc[j][r], acc[j + 1][r]);
        }
        __syncthreads();

        const bool all = now.n == now.un;
        const int which = first_piece ? 0 : 1;
        const int d4 = p.s.dim / 4;
        float* part = all ? nullptr : place(p, w, which);
        if (now.unit == 0 && crosses && threadIdx.x == 0 && (by_row || !all)) {
            const int id = now.b * p.s.rows + now.row;
            crosses[by_row ? id : w] = Cross{id, all ? -1 : w * 2 + which, cut.group_of(next_at - 1), 0};
        }
        for (int i = threadIdx.x; i < nq * d4; i += kWaves * 64) {
            const int q = i / d4, d = (i - q * d4) * 4;
            float M = kNegInf, L = 0.0f;
            float4 o = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < kWaves; ++v) M = fmaxf(M, sm[turn][v][q]);
#pragma unroll
            for (int v = 0; v < kWaves; ++v) {
                // a wave without tokens has sum and output 0 (or a NaN sum where a page was bad)
                const float f = sm[turn][v][q] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((sm[turn][v][q] - M) * p.c);
                const float4 x = *reinterpret_cast<const float4*>(&so[turn][v][q][d]);
                L += sl[turn][v][q] * f;
                o.x += x.x * f, o.y += x.y * f, o.z += x.z * f, o.w += x.w * f;
            }
            if (all) {
                const float inv = now.len <= 0 ? 0.0f : 1.0f / L;
                const int64_t at = (int64_t)now.b * p.a.Hq + now.head * p.s.group + now.q0 + q;
                *reinterpret_cast<uint2*>(p.a.out + at * p.s.dim + d) =
                    make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
                if (p.a.lse && d == 0)
                    p.a.lse[at] = now.len <= 0 ? kNegInf : lse_of(p, M, L);
            } else {
                *reinterpret_cast<float4*>(part + 32 + q * p.s.dim + d) = o;
                if (d == 0) part[2 * q] = M, part[2 * q + 1] = L;
            }
        }
        if (last) break;
        if constexpr (kOneTurn) __syncthreads();
        at = next_at;
        now = next;
        first_piece = false;
    }
}

template <int kDC, bool kFull, int kHeld, bool kForm>
void go_queries(const Args& p, bool q_fp32, hipStream_t s) {
    const dim3 grid((unsigned)p.s.groups), block(kWaves * 64);
    if (q_fp32)
        hipLaunchKernelGGL((attend_kernel<kDC, kFull, kHeld, true, kForm>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((attend_kernel<kDC, kFull, kHeld, false, kForm>), grid, block, 0, s, p);
}
// The kernels that some head_dim has: below 96 (bf16) and 192 (e4m3) width_of goes
// elsewhere, and e2m1 has none of 96.
template <int kDC, int kHeld, bool kForm>
void go_width(const Args& p, bool q_fp32, hipStream_t s) {
    constexpr bool kPart = !(kDC == 96 && kHeld != BD_E4M3) && !(kDC == 192 && kHeld == BD_E4M3);
    if (p.s.dim == kDC)
        go_queries<kDC, true, kHeld, kForm>(p, q_fp32, s);
    else if constexpr (kPart)
        go_queries<kDC, false, kHeld, kForm>(p, q_fp32, s);
}
template <int kHeld, bool kForm>
void go_held(const Args& p, bool q_fp32, hipStream_t s) {
    switch (width_of(p.s.dim, kHeld)) {
        case 64: go_width<64, kHeld, kForm>(p, q_fp32, s); break;
        case 96:
            if constexpr (kHeld != BD_E2M1) go_width<96, kHeld, kForm>(p, q_fp32, s);
            break;
        case 128: go_width<128, kHeld, kForm>(p, q_fp32, s); break;
        case 192: go_width<192, kHeld, kForm>(p, q_fp32, s); break;
        default: go_width<256, kHeld, kForm>(p, q_fp32, s);
    }
}

// One file each, so that they are built side by side.
void go_bf16(const Args& p, bool q_fp32, hipStream_t s);
void go_bf16_formed(const Args& p, bool q_fp32, hipStream_t s);
void go_e4m3(const Args& p, bool q_fp32, hipStream_t s);
void go_e4m3_formed(const Args& p, bool q_fp32, hipStream_t s);
void go_e2m1(const Args& p, bool q_fp32, hipStream_t s);
void go_e2m1_formed(const Args& p, bool q_fp32, hipStream_t s);

}  // namespace attend
}  // namespace bd
