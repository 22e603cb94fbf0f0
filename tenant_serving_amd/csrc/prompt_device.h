// Attention of several new tokens of each sequence (a prompt, or a chunk of
// one) over the paged key-value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (s_j - m)),  first <= j < last
//
// with s_j = q.k_j and c = scale log2(e), or formed scores and c = log2(e), and
// m a running maximum of s_j.  Bound by the matrix units, where the prompt is
// long, and by the exponentials between the two products: a tile's products take
// a wave 32 cycles for each of KT (KS + 2 DT) instructions, 1024 at 128 columns,
// and its weights about 1400, which the other waves' products hide for the most
// part.  8192 tokens, 64 query heads of 128 columns over 8, bf16, causal: 1055 us,
// 1040 TFLOP/s of what is not masked (a large product of matrices reaches 1170).
//
// Layout.  The rows of a tile are (token, query head) pairs of one sequence and
// one key-value head, tokens first: the heads that share keys and values share a
// tile's loads.  A wave takes 32 rows, a workgroup kWaves * 32, and goes over the
// keys kKeys at a time, which it stages in LDS as bf16, two buffers in turn:
// bf16 rows by loads that write there, codes by way of registers, converted.
//   scores  S^T [keys, rows] = K Q^T by v_mfma_f32_32x32x16_bf16, queries in
//           registers.  The A operand's row m is key 16 (m / 16) + 8 (m / 4 % 2)
//           + 4 (m / 8 % 2) + m % 4, which leaves a lane with the scores of 8
//           consecutive keys twice: 16 (r / 8) + 8 (lane / 32) + r % 8,
//   sums    O^T [dims, rows] += V^T P^T, whose B operand is just those 8 keys,
//           so weights stay in their lane.  The A operand's 8 keys of one
//           column come by ds_read_b64_tr_b16, 4 keys of 16 columns at a time.
// A row of LDS is a key: its 16-byte pieces (keys) and 64-byte pieces (values)
// are exchanged by the key's low bits, so that what a read touches at once lies
// in different banks.
// The maximum moves only when a weight would pass 2^10 (one compare and a
// ballot), so rescaling is rare and the two lanes of a row need not exchange
// theirs otherwise.  The weights enter the second product as one bf16 term: an
// output is off by half a step of bf16 of its terms at most, each its own way,
// against another half step when it is stored.
//
// Masks.  Each row has its own range of keys.  Where all rows of a wave see all
// of a key tile nothing is masked.  Elsewhere a row's scores outside its range
// are -infinity, whatever the keys hold.  Values there must not reach it either,
// and 0 times infinity or NaN would: so tiles that some row of the workgroup sees
// in part are looked through for values that are not finite as they are staged.
// Such a key's values are cleared, and added at the end to the rows that see it,
// from the cache itself.
//
// Split.  Where the rows are few a tile's keys are shared out over several
// workgroups, whose fp32 partial results a second kernel adds in order.
#pragma once

#include <type_traits>

#include "step_internal.h"

namespace bd {
namespace prompt {

constexpr float kLazy = 10.0f;      // log2: how large a weight may be before the maximum moves
constexpr float kNegInf = -__builtin_inff();
constexpr float kLeastC = 0x1p-149f;  // times it -infinity stays what it is

// A kernel's width: head_dim rounded up to 64, 96, 128, 192 or 256.
constexpr int width_of(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }
// Keys of a tile.
constexpr int keys_of(int width) { return width <= 128 ? 64 : 32; }

// Waves of a workgroup: 8 that take turns where codes are converted on the way,
// since a tile of 256 rows has half the conversions for each of them, else two
// workgroups of 4 to a CU, which drift into turns by themselves (a whole prompt
// of 8192 tokens, 64 query heads of 128 columns over 8, with 4 and with 8: bf16
// 1054 and 1081 us, e4m3 1248 and 1158, 4-bit codes capped 1790 and 1702; 64
// columns 724 and 788, with e4m3 codes 779 and 782; 192 columns 1460 and 1557,
// with codes 1647 and 1561; a chunk of 512 tokens on 32768 4-bit ones 656 and
// 574; 15 tokens on 48000 bf16 ones 48 and 63).  Formed scores at 192 columns spill
// with 8 (capped, e4m3 2094 and 2312, 4-bit codes 2211 and 2620).  At 256 columns a
// workgroup of 4 takes a CU's registers.
constexpr int waves_of(int width, int held, bool form) {
    return held == BD_BF16 || width == 64 || width == 256 || (width == 192 && form) ? 4 : 8;
}

struct Args {
    PromptArgs a;
    int32_t dim, heads, group;
    int32_t rows;                      // of a tile: 32 for each wave of a workgroup
    int32_t pg8, magic;                // groups of 8 tokens in a page
    int32_t capacity;                  // tokens a table row holds
    int32_t splits;
    uint32_t pages;                    // of the cache
    uint32_t page16, head16, token16;  // its strides in units of 16 bytes
    uint32_t page_scales, head_scales; // scale bytes of a page, of a head of it
    // what the maximum's units take to be exponents of 2, no smaller than kLeastC, and to be scores
    float c, unit;
    float times;                       // what a product takes to be a formed score
    uint32_t flip;                     // the queries' sign bits where scale is negative
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A tile: its sequence, the sequence's new tokens and length as given, and its
// first row among theirs.  Tiles are numbered over the batch, each sequence's in
// order.
struct Tile {
    int b, start, n, given;  // sequence, its first new token in the batch, new tokens, length
    int row;
    bool none;
};
__device__ __forceinline__ void tokens_of(const Args& p, int b, int* start, int* n) {
    int s0 = p.a.starts[b], s1 = p.a.starts[b + 1];
    s0 = s0 < 0 ? 0 : s0 > p.a.T ? p.a.T : s0;
    s1 = s1 < s0 ? s0 : s1 > p.a.T ? p.a.T : s1;
    *start = s0;
    *n = s1 - s0;
}
__device__ __forceinline__ int tiles_of(const Args& p, int n) { return (n * p.group + p.rows - 1) / p.rows; }
// The tile that comes `from_end`-th from the end; each wave works it out, lane l
// for `per` sequences from l per on.  Starts that rise give fewer than kTilesMost
// tiles (2^29 / 128 rows and 2^22 sequences); where they fall several sequences
// may claim the same tokens, and a lane's sum stops there, so that 64 of them fit
// 32 bits and what is found is a tile of its sequence.
constexpr int kTilesMost = 1 << 24;
__device__ __forceinline__ Tile tile_at(const Args& p, int from_end) {
    const int lane = threadIdx.x & 63;
    const int per = (p.a.B + 63) / 64, b0 = lane * per;
    int sum = 0, start = 0, n = 0, given = 0;
    for (int i = 0; i < per; ++i)
        if (b0 + i < p.a.B) {
            given = p.a.lengths[b0 + i];
            tokens_of(p, b0 + i, &start, &n);
            sum += tiles_of(p, n);
            sum = sum < kTilesMost ? sum : kTilesMost;
        }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(inc, off, 64);
        if (lane >= off) inc += o;
    }
    const int total = __builtin_amdgcn_readlane(inc, 63);
    Tile t{0, 0, 0, 0, 0, from_end >= total};
    if (t.none) return t;
    int at = total - 1 - from_end;
    // the first lane whose sequences end past it
    const int l = uni(__ffsll((unsigned long long)__ballot(inc > at)) - 1);
    at -= __builtin_amdgcn_readlane(inc - sum, l);
    t.b = l * per;
    if (per == 1) {
        start = __builtin_amdgcn_readlane(start, l);
        n = __builtin_amdgcn_readlane(n, l);
        given = __builtin_amdgcn_readlane(given, l);
    } else {
        for (;;) {
            tokens_of(p, t.b, &start, &n);
            const int tiles = tiles_of(p, uni(n));
            if (at < tiles || t.b + 1 >= p.a.B) break;
            at -= tiles;
            ++t.b;
        }
        given = p.a.lengths[t.b];
    }
    t.b = uni(t.b);
    t.start = uni(start);
    t.n = uni(n);
    t.given = uni(given);
    t.row = uni(at) * p.rows;
    return t;
}

// Partial results of a split: per tile and head, `splits` places of its rows'
// (maximum, sum) and unnormalised outputs.
__device__ __forceinline__ float* place(const Args& p, int tile, int head, int split) {
    return p.a.part + (((int64_t)tile * p.heads + head) * p.splits + split) * (p.rows * (p.dim + 2));
}

// A row's range of keys, in its sequence of `len` tokens, and its position.
struct Range {
    int lo, hi, pos;
};
__device__ __forceinline__ Range range_of(const Args& p, const Tile& t, int len, int token) {
    Range r;
    r.pos = len - t.n + token;
    r.lo = p.a.first ? p.a.first[t.start + token] : 0;
    r.hi = p.a.last ? p.a.last[t.start + token] : r.pos + 1;
    if (r.lo < 0) r.lo = 0;
    if (r.hi > len) r.hi = len;
    if (r.hi <= r.lo) r.lo = r.hi = 0;
    return r;
}

// The largest of 32 neighbouring lanes' numbers, in all of them.
template <int kCtrl>
__device__ __forceinline__ int max_dpp(int x) {
    const int o = __builtin_amdgcn_update_dpp(x, x, kCtrl, 0xf, 0xf, false);
    return o > x ? o : x;
}
__device__ __forceinline__ int max_of_half(int x) {
    x = max_dpp<0xb1>(x);   // quads: lane ^ 1
    x = max_dpp<0x4e>(x);   // lane ^ 2
    x = max_dpp<0x141>(x);  // mirrored within 8
    x = max_dpp<0x140>(x);  // mirrored within 16
    const int o = __shfl_xor(x, 16, 64);
    return o > x ? o : x;
}

// Keys [lo, hi) that some of a set of rows see, of which [all_lo, all_hi) are
// seen by all of them.
struct Keys {
    int lo, hi, all_lo, all_hi;
};
constexpr int kFar = 0x7fffffff;

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// 16 bytes for every lane, from `off` bytes behind a uniform address, written to
// LDS from `to` on, lane after lane.  (A buffer load: the compiler counts the
// LDS reads behind a global one of this kind as if they came in any order.)
__device__ __forceinline__ void load_to_lds(rsrc_t from, uint32_t off, uint32_t more, char* to) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16, off, more, 0, 0);
}

// 16 bytes of bf16 values from eight held ones.
template <int kHeld>
struct Piece;
template <>
struct Piece<BD_BF16> {
    uint4 w;
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void load(const char* at, const uint8_t*) { w = *reinterpret_cast<const uint4*>(at); }
    __device__ __forceinline__ uint4 value() const { return w; }
};
template <>
struct Piece<BD_E4M3> {
    uint2 w;
    int byte;
    __device__ __forceinline__ void zero() { w = make_uint2(0, 0), byte = 127; }
    __device__ __forceinline__ void load(const char* at, const uint8_t* scale) {
        w = *reinterpret_cast<const uint2*>(at);
        byte = *scale;
    }
    __device__ __forceinline__ uint4 value() const {
        const float s = scale_of(byte);
        return make_uint4(e4m3x2_to_bf16<false>(w.x, s), e4m3x2_to_bf16<true>(w.x, s), e4m3x2_to_bf16<false>(w.y, s),
                          e4m3x2_to_bf16<true>(w.y, s));
    }
};
template <>
struct Piece<BD_E2M1> {
    uint32_t w;
    int byte;
    __device__ __forceinline__ void zero() { w = 0, byte = 127; }
    __device__ __forceinline__ void load(const char* at, const uint8_t* scale) {
        w = *reinterpret_cast<const uint32_t*>(at);
        byte = *scale;
    }
    __device__ __forceinline__ uint4 value() const { return e2m1x8_to_bf16(w, scale_of(byte)); }
};

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(uint4 v) {
    const auto bad = [](uint32_t w) { return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u; };
    return bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
}

// How a tile lies in LDS: blocks of 8 keys by 64 columns, 128 bytes to a key, a
// key group's blocks one after another.  The 16-byte piece i of a key's part is
// at place i ^ key_swap(row), of a value's at i ^ value_swap(row): the 16 keys
// that a read of keys touches at once lie in different banks then, and so do the
// 4 values by 32 columns of a transposing read.  A block is what one wave loads
// at once, lane l its bytes 16 l .. 16 l + 15.
__device__ __forceinline__ int key_swap(int row) { return (row >> 1) & 7; }
__device__ __forceinline__ int value_swap(int row) { return (row >> 1 & 1) * 4; }

// Four of a held row's values from column d on, in fp32; `sc` is the row's scale
// byte, or that of its first group, `group` bytes before the next one's.
template <int kHeld>
__device__ __forceinline__ void four_of(const char* row, const uint8_t* sc, int group, int d, float* f) {
    uint2 w;
    if constexpr (kHeld == BD_BF16) {
        w = *reinterpret_cast<const uint2*>(row + d * 2);
    } else if constexpr (kHeld == BD_E4M3) {
        const uint32_t c = *reinterpret_cast<const uint32_t*>(row + d);
        w = make_uint2(e4m3x2_to_bf16<false>(c, scale_of(*sc)), e4m3x2_to_bf16<true>(c, scale_of(*sc)));
    } else {
        const uint32_t c = *reinterpret_cast<const uint16_t*>(row + d / 2);
        const float scale = scale_of(sc[d / kGroup4 * group]);
        w = make_uint2(e2m1x2_to_bf16<0>(c, scale), e2m1x2_to_bf16<1>(c, scale));
    }
    f[0] = __uint_as_float(w.x << 16), f[1] = __uint_as_float(w.x & 0xffff0000u);
    f[2] = __uint_as_float(w.y << 16), f[3] = __uint_as_float(w.y & 0xffff0000u);
}

// kFull: head_dim is kW and 8 tokens' rows lie within 2^31 bytes; bf16 rows of
// whole blocks go to LDS by loads that write there then.
// kWaves: 4, or 8 that take turns.
template <int kW, int kHeld, bool kForm, bool kFull, int kWaves>
__global__ __launch_bounds__(kWaves * 64, kWaves == 8 || kW <= 192 ? 2 : 1) void prompt_kernel(const Args p) {
    constexpr bool kTurns = kWaves == 8, kDma = kFull && kHeld == BD_BF16 && kW % 64 == 0;
    constexpr int kKeys = keys_of(kW), KT = kKeys / 32, KS = kW / 16, DT = kW / 32;
    constexpr int NI = (kW + 63) / 64;        // blocks of a key group
    constexpr int kGroup = NI * 1024;         // bytes of one
    constexpr int kGroups = kKeys / 8;        // of a tile
    constexpr int kBuf = kGroups * kGroup;    // bytes of a buffer of keys, or of values
    // A wave stages G groups of keys and as many of values, or where there are
    // fewer groups than waves either.
    constexpr int G = kGroups >= kWaves ? kGroups / kWaves : 1;
    constexpr bool kEither = kGroups < kWaves;
    static_assert(kEither ? 2 * kGroups == kWaves : G * kWaves == kGroups, "whole groups for every wave");
    // variables of their own, so that loads into one are not waited for where another is read
    __shared__ __attribute__((aligned(1024))) char keys0[kBuf], keys1[kBuf], values0[kBuf], values1[kBuf];
    __shared__ Keys sr[kWaves];
    __shared__ int any_odd;  // some key's values were not finite, see below

    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int head = blockIdx.x % p.heads, rest = blockIdx.x / p.heads;
    const int split = rest % p.splits, from_end = rest / p.splits;
    const Tile tile = tile_at(p, from_end);
    if (tile.none) return;
    const int given = tile.given;
    const int len = given > p.capacity || given < 0 ? 0 : given;

    // the lane's row
    const int rows = tile.n * p.group;
    const int row = tile.row + wave * 32 + col;
    const bool mine = row < rows;
    const int token = mine ? row / p.group : 0, qhead = head * p.group + (mine ? row - token * p.group : 0);

    // queries: B operand, column col, values 16 s + 8 half .. (lanes without a row take the first one's, whose results
    // are not stored)
    uint4 q[KS];
    const uint16_t* q_row = p.a.q + (tile.start + token) * p.a.qs.token + qhead * p.a.qs.head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const int d = s * 16 + half * 8;
        q[s] = *reinterpret_cast<const uint4*>(q_row + (d < p.dim ? d : 0));
    }
    const float slope = kForm && p.a.slopes ? slope_in(p.a.slopes[qhead], p.unit) : 0.0f;
    Range range{0, 0, 0};
    if (mine) range = range_of(p, tile, len, token);
    const bool sees = range.hi > range.lo;
    if (tid == 0) any_odd = 0;

    // the wave's keys and the workgroup's
    Keys own, all;
    if (!p.a.first && !p.a.last) {
        // each row's end rises with its number, and all start at 0
        const auto end_of = [&](int r) {
            const int e = len - tile.n + r / p.group + 1;
            return e < 0 ? 0 : e > len ? len : e;
        };
        const auto keys_of_rows = [&](int r0, int n) {
            if (r0 >= rows) return Keys{kFar, 0, 0, kFar};
            const int hi = end_of(r0 + n < rows ? r0 + n - 1 : rows - 1);
            return Keys{hi > 0 ? 0 : kFar, hi, 0, end_of(r0)};
        };
        own = keys_of_rows(tile.row + wave * 32, 32);
        all = keys_of_rows(tile.row, kWaves * 32);
    } else {
        own.lo = uni(-max_of_half(sees ? -range.lo : -kFar));
        own.hi = uni(max_of_half(range.hi));
        own.all_lo = uni(max_of_half(range.lo));
        own.all_hi = uni(-max_of_half(mine ? -range.hi : -kFar));
        if (lane == 0) sr[wave] = own;
        __syncthreads();
        all = sr[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) {
            const Keys k = sr[w];
            all.lo = k.lo < all.lo ? k.lo : all.lo;
            all.hi = k.hi > all.hi ? k.hi : all.hi;
            all.all_lo = k.all_lo > all.all_lo ? k.all_lo : all.all_lo;
            all.all_hi = k.all_hi < all.all_hi ? k.all_hi : all.all_hi;
        }
        all = Keys{uni(all.lo), uni(all.hi), uni(all.all_lo), uni(all.all_hi)};
    }

    // this split's key tiles, numbered from 0: n of them, the first from key j_from on
    const int base = all.lo & -kKeys;
    const int tiles = all.hi > all.lo ? (all.hi - base + kKeys - 1) / kKeys : 0;
    const int t_from = (int)((int64_t)tiles * split / p.splits), t_to = (int)((int64_t)tiles * (split + 1) / p.splits);
    const int n = t_to - t_from, j_from = base + t_from * kKeys;
    // a tile that some row of the workgroup does not see all of
    const auto edge = [&](int t) { return j_from + t * kKeys < all.all_lo || j_from + t * kKeys + kKeys > all.all_hi; };

    // Staging.  Lane l loads piece l % 8 (as the swap has it) of key l / 8 of its
    // wave's groups, in every block.  Groups before the first key and behind the
    // last are taken for these keys' groups, so that any address is one of the
    // sequence; what lies outside is masked as keys are and cleared as values are.
    const int r8 = lane >> 3, c8 = lane & 7;
    const int group0 = kEither ? wave % kGroups : wave * G;
    const bool keys_mine = !kEither || wave < kGroups, values_mine = !kEither || wave >= kGroups;
    const uint64_t token_bytes = (uint64_t)p.token16 * 16;
    constexpr int kPiece = kHeld == BD_BF16 ? 16 : kHeld == BD_E4M3 ? 8 : 4;  // bytes of eight held values
    int k_piece[G];
    uint64_t k_off[G];
    const int v_piece = c8 ^ value_swap(r8);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        k_piece[g] = c8 ^ key_swap((group0 + g) * 8 + r8);
        k_off[g] = r8 * token_bytes + k_piece[g] * kPiece;
    }
    const uint64_t v_off = r8 * token_bytes + v_piece * kPiece;
    const int32_t* table = p.a.table + tile.b * p.a.table_stride;
    const int first8 = all.lo >> 3, last8 = (all.hi - 1) >> 3;
    const auto group8 = [&](int t, int g) __attribute__((always_inline)) {
        const int g8 = ((j_from + t * kKeys) >> 3) + g;
        return g8 < first8 ? first8 : g8 > last8 ? last8 : g8;
    };
    const auto index_of = [&](int g8) __attribute__((always_inline)) {  // exact: g8 < 2^21, pg8 <= 2^9
        return (int)(((uint64_t)(uint32_t)g8 * (uint32_t)p.magic) >> 32) + (p.pg8 == 1 ? g8 : 0);
    };
    // Where a wave's group of a tile lies: byte and scale byte of its first
    // token; page 0 stands in for a bad page.  A lane works it out for one tile,
    // 64 tiles at a time.
    struct Spot {
        uint64_t to, sc;
        bool bad;
    };
    Spot spots[G];
    uint64_t bad_tiles[G];
    const auto look_up = [&](int t) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int g8 = group8(t + lane, group0 + g), idx = index_of(g8), at = (g8 - idx * p.pg8) * 8;
            uint32_t pg = (uint32_t)table[idx];
            bad_tiles[g] = __ballot(pg >= p.pages);
            if (pg >= p.pages) pg = 0;
            spots[g].to = ((uint64_t)pg * p.page16 + (uint64_t)(uint32_t)at * p.token16 + (uint64_t)(uint32_t)head * p.head16) * 16;
            spots[g].sc = (uint64_t)pg * p.page_scales + ((uint32_t)head * p.head_scales + (uint32_t)at);
        }
    };
    const auto lane64 = [](uint64_t v, int l) __attribute__((always_inline)) {
        return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), l) << 32 |
               (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, l);
    };
    const auto spot_of = [&](int t, int g) __attribute__((always_inline)) {
        const int l = t & 63;
        return Spot{lane64(spots[g].to, l), kHeld == BD_BF16 ? 0 : lane64(spots[g].sc, l), (bad_tiles[g] >> l & 1) != 0};
    };
    Piece<kHeld> kp[kDma ? 1 : G][kDma ? 1 : NI], vp[kDma ? 1 : G][kDma ? 1 : NI];
    const int scale_group = kHeld == BD_E2M1 ? p.pg8 * 8 : 0;  // scale bytes from a group of columns to the next
    const auto load = [&](const void* array, const uint8_t* scales, const Spot* x, const uint64_t* off, int same,
                          const int* piece, auto& pieces, char* to) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const char* group_at = static_cast<const char*>(array) + x[g].to;
            char* group_to = to + (group0 + g) * kGroup;
            if constexpr (kDma) {
                const rsrc_t whole = make_rsrc(group_at, 0xffffffffu);
                const uint32_t lane_off = (uint32_t)off[g * same];
#pragma unroll
                for (int i = 0; i < NI; ++i) load_to_lds(whole, lane_off, i * 128, group_to + i * 1024);
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int c = i * 8 + piece[g * same];
                    if (!(kFull && kW % 64 == 0)) pieces[g][i].zero();
                    if ((kFull && kW % 64 == 0) || c * 8 < p.dim)
                        pieces[g][i].load(group_at + off[g * same] + i * 8 * kPiece, scales + x[g].sc + r8 + c / 4 * scale_group);
                }
            }
        }
    };
    const auto store = [&](auto& pieces, char* to) __attribute__((always_inline)) {
        if constexpr (!kDma) {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    *reinterpret_cast<uint4*>(to + (group0 + g) * kGroup + i * 1024 + lane * 16) = pieces[g][i].value();
        }
    };
    // Keys that have come for a bad page: NaN, as the scores of those that see them.
    const auto spoil = [&](const Spot* x, char* keys) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < G; ++g)
            if (x[g].bad) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    *reinterpret_cast<uint4*>(keys + (group0 + g) * kGroup + i * 1024 + lane * 16) =
                        make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
            }
    };
    // Values of tile t that have come, where some row does not see all of it or
    // a page is bad: what is outside the keys is cleared, and so are keys whose
    // values are not finite, which are made up for at the end.
    const auto clean = [&](int t, const Spot* x, char* values) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int r = (group0 + g) * 8 + r8, j = j_from + t * kKeys + r;
            uint4* at = reinterpret_cast<uint4*>(values + (group0 + g) * kGroup + lane * 16);
            bool odd = false;
#pragma unroll
            for (int i = 0; i < NI; ++i) odd |= not_finite(at[i * 64]);
            const uint64_t rows_odd = __ballot(odd) >> (lane & 56) & 0xff;  // of the key's eight lanes
            const bool out = j < all.lo || j >= all.hi || x[g].bad;
            if (out || rows_odd) {
#pragma unroll
                for (int i = 0; i < NI; ++i) at[i * 64] = make_uint4(0, 0, 0, 0);
                if (!out) any_odd = 1;
            }
        }
    };

    f32x16_t o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    // The weights are 2^(c s - mc), mc = c m rounded: one operation before the
    // exponential.  What the rounding adds to all of them, c m - mc, is exact in
    // fp32 (`rest_c`) and taken out where the sums change their maximum or end.
    // Where mc is so large that this could pass fp32's range (`careful`), the
    // difference to m comes first.
    float m = kNegInf, l = 0.0f, mc = 0.0f, rest_c = 0.0f;
    bool careful = false;
    const float c = p.c;

    // where the lane reads keys and values; what a step of the products adds is the same for all lanes
    const int key = (col & 16) + (col >> 2 & 1) * 8 + (col >> 3 & 1) * 4 + (col & 3);
    const int k_base = (key >> 3) * kGroup + (key & 7) * 128 + (half ^ key_swap(key)) * 16;
    const int l16 = lane & 15;
    const int v_row = l16 >> 2;
    const int v_base = half * kGroup + v_row * 128 + value_swap(v_row) * 16 + (lane >> 4 & 1) * 32 + (l16 & 3) * 8;

    f32x16_t s[KT];     // scores of the tile in work
    uint4 pw[KT * 2];   // its weights, 8 consecutive keys each
#pragma unroll
    for (int i = 0; i < KT * 2; ++i) pw[i] = make_uint4(0, 0, 0, 0);

    // The matrix products' turn: the sums of the tile before and the scores of
    // this one, in a row of steps of one product each, whose A operands are read
    // kAhead steps before.
    constexpr int kSums = KT * 2 * DT, kScores = KT * KS, kAhead = 6;
    const auto value_at = [&](const char* values, int step) __attribute__((always_inline)) {
        const int i = step / DT, dt = step % DT;
        const char* at = values + (v_base ^ (dt % 2 * 64)) + dt / 2 * 1024 + i * 2 * kGroup;
        const uint2 a0 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at));
        const uint2 a1 = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 512)));
        return make_uint4(a0.x, a0.y, a1.x, a1.y);
    };
    const auto key_at = [&](const char* keys, int step) __attribute__((always_inline)) {
        const int kt = step / KS, i = step % KS;
        return *reinterpret_cast<const uint4*>(keys + (k_base ^ (i % 4 * 32)) + i / 4 * 1024 + kt * 4 * kGroup);
    };
    const auto products = [&](auto scores, const char* keys, const char* values) __attribute__((always_inline)) {
        constexpr int kFrom = 0, kTo = decltype(scores)::value ? kSums + kScores : kSums;
        if (kTurns) __builtin_amdgcn_s_setprio(1);
        const auto fetch = [&](int step) __attribute__((always_inline)) {
            return step < kSums ? value_at(values, step) : key_at(keys, step - kSums);
        };
        uint4 a[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) a[i] = fetch(kFrom + i);
#pragma unroll
        for (int step = kFrom; step < kTo; ++step) {
            const bf16x8_t x = as_bf16x8(a[(step - kFrom) % kAhead]);
            if (step < kSums) {
                o[step % DT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, as_bf16x8(pw[step / DT]), o[step % DT], 0, 0, 0);
            } else {
                const int kt = (step - kSums) / KS, i = (step - kSums) % KS;
                if (i == 0) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) s[kt][r] = 0.0f;
                }
                s[kt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, as_bf16x8(q[i]), s[kt], 0, 0, 0);
            }
            if (step + kAhead < kTo) a[(step - kFrom) % kAhead] = fetch(step + kAhead);
        }
        // in just this order
#pragma unroll
        for (int i = 0; i < kAhead; ++i) kFrom + i < kSums ? __builtin_amdgcn_sched_group_barrier(0x100, 2, 0) : __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
#pragma unroll
        for (int step = kFrom; step < kTo; ++step) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            if (step + kAhead < kTo) step + kAhead < kSums ? __builtin_amdgcn_sched_group_barrier(0x100, 2, 0) : __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        if (kTurns) __builtin_amdgcn_s_setprio(0);
    };

    // The weights of tile t from its scores.
    const auto weights = [&](int t) __attribute__((always_inline)) {
        const int j0 = j_from + t * kKeys;
        float sc[KT * 16];
#pragma unroll
        for (int i = 0; i < KT * 16; ++i) sc[i] = s[i / 16][i % 16];
        if constexpr (kForm) {
            if (p.a.cap > 0.0f) {
#pragma unroll
                for (int i = 0; i < KT * 2; ++i) cap_scores<8>(sc + 8 * i, p.times);
            } else {
#pragma unroll
                for (int i = 0; i < KT * 16; ++i) sc[i] *= p.times;
            }
            if (p.a.slopes) {
                const float far = (float)(range.pos - j0 - 8 * half);
#pragma unroll
                for (int i = 0; i < KT * 16; ++i)
                    sc[i] = __builtin_fmaf(-slope, __builtin_fabsf(far - (float)(i / 8 * 16 + i % 8)), sc[i]);
            }
        }
        if (j0 < own.all_lo || j0 + kKeys > own.all_hi) {
            // a bit for each of the tile's keys that the row sees, then of the lane's own; two operations for each score
            const int lo = range.lo - j0, hi = range.hi - j0;
            const auto below = [](int n) __attribute__((always_inline)) {
                return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
            };
            const uint64_t seen = below(hi) & ~below(lo);
            const uint32_t bits = __builtin_amdgcn_perm((uint32_t)(seen >> 32), (uint32_t)seen, half ? 0x07050301u : 0x06040200u);
#pragma unroll
            for (int i = 0; i < KT * 16; ++i) {
                const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)bits, i, 1);
                sc[i] = __uint_as_float((__float_as_uint(sc[i]) & keep) | (0xff800000u & ~keep));
            }
        }
        float mx = sc[0];
#pragma unroll
        for (int i = 1; i < KT * 16; ++i) mx = fmaxf(mx, sc[i]);
        if (__ballot((mx - m) * c > kLazy)) {
            mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
            const float up = fmaxf(m, mx);
            const float to = up == kNegInf ? 0.0f : up;
            mc = to * c;
            careful = __ballot(!(__builtin_fabsf(mc) < 16777216.0f)) != 0;
            const float was = rest_c;
            rest_c = careful ? 0.0f : __builtin_fmaf(to, c, -mc);
            const float f = __builtin_amdgcn_exp2f((m - to) * c + (rest_c - was));
            m = up;
            l *= f;
#pragma unroll
            for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int r = 0; r < 16; ++r) o[i][r] *= f;
        }
        if (careful) {
            const float mm = m == kNegInf ? 0.0f : m;
#pragma unroll
            for (int i = 0; i < KT * 16; ++i) sc[i] = __builtin_amdgcn_exp2f((sc[i] - mm) * c);
        } else {
#pragma unroll
            for (int i = 0; i < KT * 16; ++i) sc[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], c, -mc));
        }
#pragma unroll
        for (int i = 0; i < KT * 2; ++i) {
#pragma unroll
            for (int r = 0; r < 8; ++r) l += sc[8 * i + r];
            pw[i] = narrow_bf16x8(sc + 8 * i);
        }
    };

#pragma unroll
    for (int i = 0; i < KS; ++i) {
        q[i].x ^= p.flip, q[i].y ^= p.flip, q[i].z ^= p.flip, q[i].w ^= p.flip;
        if (i * 16 + half * 8 >= p.dim) q[i] = make_uint4(0, 0, 0, 0);
    }
    // round 0 has no tile before it: its weights and values are zeros
    for (int i = tid * 16; i < kBuf; i += kWaves * 1024) *reinterpret_cast<uint4*>(values1 + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();  // the mark is clear

    // Round t: the sums of tile t - 1 and the scores of tile t (products), then
    // its weights, while the keys of tile t + 1 and the values of tile t come.
    // With 8 waves the second four are half a round behind, so that of the two
    // waves of a SIMD one has products and the other weights to work on; their
    // share of the staging is not, so it starts and ends half a round earlier
    // in theirs.
    const bool late = kTurns && wave >= kWaves / 2;
    Spot next[G], now[G];
    if (n > 0) {
        look_up(0);
#pragma unroll
        for (int g = 0; g < G; ++g) next[g] = spot_of(0, g);
        if (keys_mine) {
            load(p.a.kv.k, p.a.kv.k_scales, next, k_off, 1, k_piece, kp, keys0);
            if constexpr (kDma) __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
            store(kp, keys0);
            spoil(next, keys0);
        }
    }
    __syncthreads();

    const auto begin = [&](int t, char* keys_to, char* values_to) __attribute__((always_inline)) {
#pragma unroll
        for (int g = 0; g < G; ++g) now[g] = next[g];
        if (t + 1 < n) {
            if (((t + 1) & 63) == 0) look_up(t + 1);
#pragma unroll
            for (int g = 0; g < G; ++g) next[g] = spot_of(t + 1, g);
            if (keys_mine) load(p.a.kv.k, p.a.kv.k_scales, next, k_off, 1, k_piece, kp, keys_to);
        }
        if (t < n && values_mine) load(p.a.kv.v, p.a.kv.v_scales, now, &v_off, 0, &v_piece, vp, values_to);
    };
    const auto end = [&](int t, char* keys_to, char* values_to) __attribute__((always_inline)) {
        if constexpr (kDma) __builtin_amdgcn_s_waitcnt(0x0f70);
        if (t + 1 < n && keys_mine) {
            store(kp, keys_to);
            spoil(next, keys_to);
        }
        if (t < n && values_mine) {
            store(vp, values_to);
            bool bad = edge(t);
#pragma unroll
            for (int g = 0; g < G; ++g) bad |= now[g].bad;
            if (bad) clean(t, now, values_to);
        }
    };
    // Where waves meet, those that have just staged wait for their loads and
    // writes first; the others' loads stay on their way, which a plain barrier
    // would wait for too.
    const auto meet = [&](bool staged) __attribute__((always_inline)) {
        asm volatile("" ::: "memory");
        if (staged) __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // keys0 and values0 have the even tiles.  A wave none of whose rows sees a
    // key only stages.
    const bool idle = own.hi == 0;
    const auto round = [&](int t, char* keys, char* keys_to, char* values, char* values_to) __attribute__((always_inline)) {
        if (!late) begin(t, keys_to, values_to);
        if (!idle) products(std::true_type{}, keys, values);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kTurns) {
            if (late) end(t, keys_to, values_to);
            meet(late);
            if (late) begin(t + 1, keys, values);
        }
        if (!idle) weights(t);
        __builtin_amdgcn_sched_barrier(0);
        if (!late) end(t, keys_to, values_to);
        if (!late || t + 1 < n) meet(!late);
    };
    if (n > 0) {
        if (late) {
            begin(0, keys1, values0);
            meet(false);
        }
        int t = 0;
        for (;;) {
            round(t, keys0, keys1, values1, values0);
            if (++t >= n) break;
            round(t, keys1, keys0, values0, values1);
            if (++t >= n) break;
        }
        // the last tile's sums, whose values have been there since the last round's staging
        if (!idle) products(std::false_type{}, nullptr, n & 1 ? values0 : values1);
    }

    // Keys that were cleared above: what they add to the rows that see them, from
    // the cache itself, one key after another and 32 columns at a time.
    if (uni(any_odd)) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
#pragma nounroll
            for (int at = 0; at < n * kKeys; ++at) {
                const int t = at / kKeys, j = j_from + at;
                if (!edge(t) || j < all.lo || j >= all.hi) continue;
                const int idx = index_of(j >> 3), place = j - idx * p.pg8 * 8;
                const uint32_t pg = (uint32_t)uni(table[idx]);
                if (pg >= p.pages) continue;
                const uint64_t to = ((uint64_t)pg * p.page16 + (uint64_t)(uint32_t)place * p.token16 +
                                     (uint64_t)(uint32_t)head * p.head16) * 16;
                const uint64_t sc = (uint64_t)pg * p.page_scales + ((uint32_t)head * p.head_scales + (uint32_t)place);
                const char* k = static_cast<const char*>(p.a.kv.k) + to;
                const char* v = static_cast<const char*>(p.a.kv.v) + to;
                float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (lane * 4 < p.dim) four_of<kHeld>(v, p.a.kv.v_scales + sc, scale_group, lane * 4, f);
                if (!__ballot((f[0] * 0.0f + f[1] * 0.0f) + (f[2] * 0.0f + f[3] * 0.0f) != 0.0f)) continue;
                float x = 0.0f;
#pragma nounroll
                for (int d = half * 4; d < p.dim; d += 8) {
                    const uint2 w = *reinterpret_cast<const uint2*>(q_row + d);
                    four_of<kHeld>(k, p.a.kv.k_scales + sc, scale_group, d, f);
                    x = __builtin_fmaf(f[0], __uint_as_float((w.x ^ p.flip) << 16), x);
                    x = __builtin_fmaf(f[1], __uint_as_float((w.x ^ p.flip) & 0xffff0000u), x);
                    x = __builtin_fmaf(f[2], __uint_as_float((w.y ^ p.flip) << 16), x);
                    x = __builtin_fmaf(f[3], __uint_as_float((w.y ^ p.flip) & 0xffff0000u), x);
                }
                x += __shfl_xor(x, 32, 64);
                if constexpr (kForm) {
                    if (p.a.cap > 0.0f)
                        cap_scores<1>(&x, p.times);
                    else
                        x *= p.times;
                    x = __builtin_fmaf(-slope, __builtin_fabsf((float)(range.pos - j)), x);
                }
                const float w = __builtin_amdgcn_exp2f(careful ? (x - (m == kNegInf ? 0.0f : m)) * c : __builtin_fmaf(x, c, -mc));
                const bool seen = j >= range.lo && j < range.hi;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int d = dt * 32 + b * 8 + half * 4;
                    if (d < p.dim) four_of<kHeld>(v, p.a.kv.v_scales + sc, scale_group, d, f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = o[dt][4 * b + e];
                        o[dt][4 * b + e] = seen ? __builtin_fmaf(w, f[e], y) : y;
                    }
                }
            }
        }
    }

    l += __shfl_xor(l, 32, 64);
    const float fix = __builtin_amdgcn_exp2f(-rest_c);
    if (!mine) return;
    const int64_t at = (int64_t)(tile.start + token) * p.a.Hq + qhead;
    if (p.splits > 1) {
        float* part = place(p, from_end, head, split);
        const int r = wave * 32 + col;
        if (half == 0) part[2 * r] = m, part[2 * r + 1] = l * fix;
        float* to = part + 2 * p.rows + r * p.dim + half * 4;
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                if (dt * 32 + x * 8 + half * 4 < p.dim)
                    *reinterpret_cast<float4*>(to + dt * 32 + x * 8) =
                        make_float4(o[dt][4 * x] * fix, o[dt][4 * x + 1] * fix, o[dt][4 * x + 2] * fix, o[dt][4 * x + 3] * fix);
        return;
    }
    float inv = sees ? 1.0f / l : 0.0f;
    if (given > p.capacity) inv = __builtin_nanf("");
    uint16_t* to = p.a.out + at * p.dim + half * 4;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (dt * 32 + x * 8 + half * 4 < p.dim)
                *reinterpret_cast<uint2*>(to + dt * 32 + x * 8) =
                    make_uint2(pack_bf16x2(o[dt][4 * x] * inv, o[dt][4 * x + 1] * inv),
                               pack_bf16x2(o[dt][4 * x + 2] * inv, o[dt][4 * x + 3] * inv));
    if (p.a.lse && half == 0) {
        const float v = __builtin_fmaf(m, p.unit, __builtin_amdgcn_logf(l * fix) * 0.69314718055994531f);
        p.a.lse[at] = given > p.capacity ? __builtin_nanf("") : sees ? v : kNegInf;
    }
}

template <int kW, int kHeld, bool kForm>
void go_width(const Args& p, unsigned groups, hipStream_t s) {
    constexpr int kWaves = waves_of(kW, kHeld, kForm);
    const dim3 grid(groups), block(kWaves * 64);
    if (p.dim == kW && p.token16 < (1u << 24))
        hipLaunchKernelGGL((prompt_kernel<kW, kHeld, kForm, true, kWaves>), grid, block, 0, s, p);
    else
        hipLaunchKernelGGL((prompt_kernel<kW, kHeld, kForm, false, kWaves>), grid, block, 0, s, p);
}
template <int kHeld, bool kForm>
void go(const Args& p, unsigned groups, hipStream_t s) {
    switch (width_of(p.dim)) {
        case 64: go_width<64, kHeld, kForm>(p, groups, s); break;
        case 96: go_width<96, kHeld, kForm>(p, groups, s); break;
        case 128: go_width<128, kHeld, kForm>(p, groups, s); break;
        case 192: go_width<192, kHeld, kForm>(p, groups, s); break;
        default: go_width<256, kHeld, kForm>(p, groups, s);
    }
}

// One file each, so that they are built side by side.
void go_bf16(const Args& p, unsigned groups, hipStream_t s);
void go_bf16_formed(const Args& p, unsigned groups, hipStream_t s);
void go_e4m3(const Args& p, unsigned groups, hipStream_t s);
void go_e4m3_formed(const Args& p, unsigned groups, hipStream_t s);
void go_e2m1(const Args& p, unsigned groups, hipStream_t s);
void go_e2m1_formed(const Args& p, unsigned groups, hipStream_t s);

}  // namespace prompt
}  // namespace bd
