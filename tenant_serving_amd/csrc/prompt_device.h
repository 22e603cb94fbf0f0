// Attention of several new tokens of each sequence (a prompt, or a chunk of
// one) over the paged key-value cache.
//
//   out = sum_j p_j v_j / sum_j p_j,   p_j = 2^(c (s_j - m)),  first <= j < last
//
// with s_j = q.k_j and c = scale log2(e), or formed scores and c = log2(e), and
// m a running maximum of s_j.  Bound by the matrix units, where the prompt is
// long, and by the exponentials between the two products.
//
// Layout.  The rows of a tile are (token, query head) pairs of one sequence and
// one key-value head, tokens first: the heads that share keys and values share a
// tile's loads.  A wave takes 32 rows, a workgroup kWaves * 32, and goes over the
// keys kKeys at a time, which it stages in LDS as bf16, codes converted on the
// way, two buffers in turn.
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
// in part are looked through for values that are not finite as they are staged,
// and the keys that hold some are taken apart from the product, by a sum that
// leaves out the rows that do not see them.
//
// Split.  Where the rows are few a tile's keys are shared out over several
// workgroups, whose fp32 partial results a second kernel adds in order.
#pragma once

#include "step_internal.h"

namespace bd {
namespace prompt {

constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kRows = kWaves * 32;  // of a tile
constexpr float kLazy = 10.0f;      // log2: how large a weight may be before the maximum moves
constexpr float kNegInf = -__builtin_inff();
constexpr float kLeastC = 0x1p-149f;  // times it -infinity stays what it is

// A kernel's width: head_dim rounded up to 64, 96, 128, 192 or 256.
constexpr int width_of(int dim) { return dim <= 64 ? 64 : dim <= 96 ? 96 : dim <= 128 ? 128 : dim <= 192 ? 192 : 256; }
// Keys of a tile: two buffers of keys and values in half a CU's LDS.
constexpr int keys_of(int width) { return width <= 128 ? 64 : 32; }

struct Args {
    PromptArgs a;
    int32_t dim, heads, group;
    int32_t pg8, magic;                // groups of 8 tokens in a page
    int32_t capacity;                  // tokens a table row holds
    int32_t splits;
    uint32_t pages;                    // of the cache
    uint32_t page16, head16, token16;  // its strides in units of 16 bytes
    uint32_t page_scales, head_scales; // scale bytes of a page, of a head of it
    float c;                           // what the maximum's units take to be exponents of 2
    float unit;                        // what they take to be scores
    uint32_t flip;                     // the queries' sign bits where scale is negative
};

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A tile: its sequence, the sequence's new tokens, and its first row among
// theirs.  Tiles are numbered over the batch, each sequence's in order.
struct Tile {
    int b, start, n;  // sequence, its first new token in the batch, new tokens
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
__device__ __forceinline__ int tiles_of(const Args& p, int n) { return (n * p.group + kRows - 1) / kRows; }
// The tile that comes `from_end`-th from the end; each wave works it out.
__device__ __forceinline__ Tile tile_at(const Args& p, int from_end) {
    const int lane = threadIdx.x & 63;
    const int per = (p.a.B + 63) / 64, b0 = lane * per;
    int sum = 0, start, n;
    for (int i = 0; i < per; ++i)
        if (b0 + i < p.a.B) {
            tokens_of(p, b0 + i, &start, &n);
            sum += tiles_of(p, n);
        }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(inc, off, 64);
        if (lane >= off) inc += o;
    }
    const int total = uni(__shfl(inc, 63, 64));
    Tile t{0, 0, 0, 0, from_end >= total};
    if (t.none) return t;
    int at = total - 1 - from_end;
    // the first lane whose sequences end past it
    const int l = __ffsll((unsigned long long)__ballot(inc > at)) - 1;
    at -= uni(__shfl(inc - sum, l, 64));
    t.b = l * per;
    for (;;) {
        tokens_of(p, t.b, &start, &n);
        const int tiles = tiles_of(p, uni(n));
        if (at < tiles || t.b + 1 >= p.a.B) break;
        at -= tiles;
        ++t.b;
    }
    t.b = uni(t.b);
    t.start = uni(start);
    t.n = uni(n);
    t.row = uni(at) * kRows;
    return t;
}

// Partial results of a split: per tile and head, `splits` places of kRows rows'
// (maximum, sum) and unnormalised outputs.
__device__ __forceinline__ float* place(const Args& p, int tile, int head, int split) {
    return p.a.part + (((int64_t)tile * p.heads + head) * p.splits + split) * (kRows * (p.dim + 2));
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

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;

// 16 bytes for every lane, written to LDS from `to` on, lane after lane.
__device__ __forceinline__ void load_to_lds(const char* from, char* to) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)from,
                                     (__attribute__((address_space(3))) void*)to, 16, 0, 0);
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

// kDma: bf16 rows of full width go to LDS by loads that write there.
template <int kW, int kHeld, bool kForm, bool kDma>
__global__ __launch_bounds__(kThreads, kW <= 192 ? 2 : 1) void prompt_kernel(const Args p) {
    constexpr int kKeys = keys_of(kW), KT = kKeys / 32, KS = kW / 16, DT = kW / 32;
    constexpr int NI = (kW + 63) / 64;             // blocks of a key group
    constexpr int kGroup = NI * 1024;              // bytes of one
    constexpr int kBuf = kKeys / 8 * kGroup;       // bytes of a buffer of keys, or of values
    constexpr int G = kKeys / 8 / kWaves;          // key groups that a wave stages
    static_assert(G * kWaves * 8 == kKeys, "whole groups for every wave");
    // two variables, so that the loads into one are not waited for where the other is read
    __shared__ __attribute__((aligned(1024))) char smem0[2 * kBuf], smem1[2 * kBuf];
    __shared__ int sr[4][kWaves];
    // of the tile in work and the two after it: whether there are any, keys with values not finite, keys of bad pages
    __shared__ uint32_t sbad[3][5];

    const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int head = blockIdx.x % p.heads, rest = blockIdx.x / p.heads;
    const int split = rest % p.splits, from_end = rest / p.splits;
    const Tile tile = tile_at(p, from_end);
    if (tile.none) return;
    const int given = uni(p.a.lengths[tile.b]);
    const int len = given > p.capacity || given < 0 ? 0 : given;

    // the lane's row
    const int row = tile.row + wave * 32 + col;
    const bool mine = row < tile.n * p.group;
    const int token = mine ? row / p.group : 0, qhead = head * p.group + (mine ? row - token * p.group : 0);
    Range range{0, 0, 0};
    if (mine) range = range_of(p, tile, len, token);
    const float slope = kForm && p.a.slopes && mine ? p.a.slopes[qhead] : 0.0f;

    // the wave's keys [w_lo, w_hi), of which [e_lo, e_hi) are seen by all its rows; then the workgroup's
    const bool sees = range.hi > range.lo;
    int w_lo = sees ? range.lo : 0x7fffffff, w_hi = range.hi;
    int e_lo = range.lo, e_hi = mine ? range.hi : 0x7fffffff;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        int o = __shfl_xor(w_lo, off, 64);
        w_lo = o < w_lo ? o : w_lo;
        o = __shfl_xor(w_hi, off, 64);
        w_hi = o > w_hi ? o : w_hi;
        o = __shfl_xor(e_lo, off, 64);
        e_lo = o > e_lo ? o : e_lo;
        o = __shfl_xor(e_hi, off, 64);
        e_hi = o < e_hi ? o : e_hi;
    }
    w_lo = uni(w_lo), w_hi = uni(w_hi), e_lo = uni(e_lo), e_hi = uni(e_hi);
    if (lane == 0) sr[0][wave] = w_lo, sr[1][wave] = w_hi, sr[2][wave] = e_lo, sr[3][wave] = e_hi;
    if (tid < 15) (&sbad[0][0])[tid] = 0;
    __syncthreads();
    int k_lo = sr[0][0], k_hi = sr[1][0], g_lo = sr[2][0], g_hi = sr[3][0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
        k_lo = sr[0][w] < k_lo ? sr[0][w] : k_lo;
        k_hi = sr[1][w] > k_hi ? sr[1][w] : k_hi;
        g_lo = sr[2][w] > g_lo ? sr[2][w] : g_lo;
        g_hi = sr[3][w] < g_hi ? sr[3][w] : g_hi;
    }
    k_lo = uni(k_lo), k_hi = uni(k_hi), g_lo = uni(g_lo), g_hi = uni(g_hi);

    // this split's key tiles
    const int base = k_lo & -kKeys;
    const int tiles = k_hi > k_lo ? (k_hi - base + kKeys - 1) / kKeys : 0;
    const int t_from = (int)((int64_t)tiles * split / p.splits), t_to = (int)((int64_t)tiles * (split + 1) / p.splits);

    // queries: B operand, column col, values 16 s + 8 half ..
    uint4 q[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        q[s] = make_uint4(0, 0, 0, 0);
        const int d = s * 16 + half * 8;
        if (mine && d < p.dim) {
            q[s] = *reinterpret_cast<const uint4*>(p.a.q + (tile.start + token) * p.a.qs.token + qhead * p.a.qs.head + d);
            q[s].x ^= p.flip, q[s].y ^= p.flip, q[s].z ^= p.flip, q[s].w ^= p.flip;
        }
    }

    // Staging.  A wave takes G groups of 8 keys; lane l loads piece l % 8 (as
    // the swap has it) of key l / 8, in every block.  Groups before the first
    // key and behind the last are taken for these keys' groups, so that any
    // address is one of the sequence; what lies outside is masked as keys are
    // and cleared as values are.
    const int r8 = lane >> 3, c8 = lane & 7;
    const uint64_t token_bytes = (uint64_t)p.token16 * 16;
    constexpr int kPiece = kHeld == BD_BF16 ? 16 : kHeld == BD_E4M3 ? 8 : 4;  // bytes of eight held values
    int k_piece[G];
    uint64_t k_off[G], v_off;
    const int v_piece = c8 ^ value_swap(r8);
#pragma unroll
    for (int g = 0; g < G; ++g) {
        k_piece[g] = c8 ^ key_swap((wave * G + g) * 8 + r8);
        k_off[g] = r8 * token_bytes + k_piece[g] * kPiece;
    }
    v_off = r8 * token_bytes + v_piece * kPiece;
    Piece<kHeld> kp[kDma ? 1 : G][kDma ? 1 : NI], vp[kDma ? 1 : G][kDma ? 1 : NI];
    int page[G];        // of the tile after the one in flight, still on their way
    uint32_t lost = 0;  // groups in flight whose page is a bad one
    const int32_t* table = p.a.table + tile.b * p.a.table_stride;
    const int first8 = k_lo >> 3, last8 = (k_hi - 1) >> 3;
    const auto group8 = [&](int t, int g) {
        const int g8 = (base >> 3) + t * (kKeys / 8) + wave * G + g;
        return g8 < first8 ? first8 : g8 > last8 ? last8 : g8;
    };
    const auto index_of = [&](int g8) {  // exact: g8 < 2^21, pg8 <= 2^9
        return (int)(((uint64_t)(uint32_t)g8 * (uint32_t)p.magic) >> 32) + (p.pg8 == 1 ? g8 : 0);
    };
    const auto look_up = [&](int t) {
#pragma unroll
        for (int g = 0; g < G; ++g) page[g] = table[index_of(group8(t, g))];
    };
    const auto load = [&](int t, char* smem) {
        lost = 0;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int g8 = group8(t, g), at = (g8 - index_of(g8) * p.pg8) * 8;
            uint32_t pg = (uint32_t)uni(page[g]);
            if (pg >= p.pages) {
                lost |= 1u << g;
                pg = 0;
            }
            const uint64_t to = ((uint64_t)pg * p.page16 + (uint64_t)(uint32_t)at * p.token16 +
                                 (uint64_t)(uint32_t)head * p.head16) * 16;
            const char* k = static_cast<const char*>(p.a.kv.k) + to;
            const char* v = static_cast<const char*>(p.a.kv.v) + to;
            if constexpr (kDma) {
                char* ks = smem + (wave * G + g) * kGroup;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    load_to_lds(k + k_off[g] + i * 128, ks + i * 1024);
                    load_to_lds(v + v_off + i * 128, ks + kBuf + i * 1024);
                }
            } else {
                const uint64_t sc = (uint64_t)pg * p.page_scales + ((uint32_t)head * p.head_scales + (uint32_t)at);
                const uint8_t* k_sc = p.a.kv.k_scales + sc + r8;
                const uint8_t* v_sc = p.a.kv.v_scales + sc + r8;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    kp[g][i].zero();
                    vp[g][i].zero();
                    const int k_at = i * 8 + k_piece[g], v_at = i * 8 + v_piece;
                    const int group = kHeld == BD_E2M1 ? p.pg8 * 8 : 0;  // scale bytes of a group of columns
                    if (k_at * 8 < p.dim) kp[g][i].load(k + k_off[g] + i * 8 * kPiece, k_sc + k_at / 4 * group);
                    if (v_at * 8 < p.dim) vp[g][i].load(v + v_off + i * 8 * kPiece, v_sc + v_at / 4 * group);
                }
            }
        }
    };
    // The tile in flight, when it has come: into LDS, and where some row sees
    // part of it only, what is outside the keys cleared and values that are not
    // finite marked.
    const auto stage = [&](int t, char* smem, int turn) {
        const int j0 = base + t * kKeys;
        const bool edge = j0 < g_lo || j0 + kKeys > g_hi;
        char* ks = smem + wave * (G * kGroup) + lane * 16;
        if constexpr (kDma) {
            __builtin_amdgcn_s_waitcnt(0x0f70);  // vmcnt(0)
        } else {
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    *reinterpret_cast<uint4*>(ks + g * kGroup + i * 1024) = kp[g][i].value();
                    *reinterpret_cast<uint4*>(ks + kBuf + g * kGroup + i * 1024) = vp[g][i].value();
                }
        }
        if (edge || lost) {
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int r = (wave * G + g) * 8 + r8, j = j0 + r;
                const bool in = j >= k_lo && j < k_hi, gone = lost >> g & 1;
                uint32_t* bad = sbad[turn];
                bool odd = false;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    uint4* v = reinterpret_cast<uint4*>(ks + kBuf + g * kGroup + i * 1024);
                    if (!in || gone)
                        *v = make_uint4(0, 0, 0, 0);
                    else
                        odd |= not_finite(*v);
                }
                if (in && (odd || gone)) {
                    atomicOr(&bad[(gone ? 3 : 1) + (r >> 5)], 1u << (r & 31));
                    bad[0] = 1;
                }
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
    // fp32 (`rest`) and taken out where the sums change their maximum or end.
    // Where mc is so large that this could pass fp32's range (`careful`), the
    // difference to m comes first.
    float m = kNegInf, l = 0.0f, mc = 0.0f, rest_c = 0.0f;
    bool careful = false;
    const float c = p.c, times = kForm ? __builtin_fabsf(p.a.scale) : 1.0f;

    // where the lane reads keys and values; what a step of the products adds is the same for all lanes
    const int key = (col & 16) + (col >> 2 & 1) * 8 + (col >> 3 & 1) * 4 + (col & 3);
    const int k_base = (key >> 3) * kGroup + (key & 7) * 128 + (half ^ key_swap(key)) * 16;
    const int l16 = lane & 15;
    const int v_row = l16 >> 2;
    const int v_base = half * kGroup + v_row * 128 + value_swap(v_row) * 16 + (lane >> 4 & 1) * 32 + (l16 & 3) * 8;

    if (t_from < t_to) {
        look_up(t_from);
        load(t_from, smem0);
        look_up(t_from + 1);
        stage(t_from, smem0, 0);
    }
    __syncthreads();

    int turn = 0;
    // One key tile, in `smem`, while the next one comes into `other`.
    const auto work = [&](int t, char* smem, char* other) {
        const bool more = t + 1 < t_to;
        if (more) {
            load(t + 1, other);
            look_up(t + 2);
        }
        const int j0 = base + t * kKeys;
        const bool here = j0 < w_hi && j0 + kKeys > w_lo;  // this wave has rows that see some of it
        const uint32_t marked = uni(sbad[turn][0]);
        const int next_turn = turn == 2 ? 0 : turn + 1;
        if (tid < 5) sbad[next_turn == 2 ? 0 : next_turn + 1][tid] = 0;
        const char* ks = smem;
        const char* vs = ks + kBuf;
        uint4 pw[KT * 2];  // weights, 8 consecutive keys each
        if (here) {
            float sc[KT * 16];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                f32x16_t s;
#pragma unroll
                for (int r = 0; r < 16; ++r) s[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    const uint4 a = *reinterpret_cast<const uint4*>(ks + (k_base ^ (i % 4 * 32)) + i / 4 * 1024 + kt * 4 * kGroup);
                    s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(a), as_bf16x8(q[i]), s, 0, 0, 0);
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) sc[kt * 16 + r] = s[r];
            }
            if constexpr (kForm) {
#pragma unroll
                for (int i = 0; i < KT * 16; ++i) sc[i] *= times;
                if (p.a.cap > 0.0f) {
#pragma unroll
                    for (int i = 0; i < KT * 2; ++i) cap_scores<8>(sc + 8 * i, p.a.cap);
                }
                if (p.a.slopes) {
                    const int far = range.pos - j0 - 8 * half;
#pragma unroll
                    for (int i = 0; i < KT * 16; ++i)
                        sc[i] = __builtin_fmaf(-slope, __builtin_fabsf((float)(far - (i / 8 * 16 + i % 8))), sc[i]);
                }
            }
            if (marked) {
                const uint32_t no0 = sbad[turn][3] >> 8 * half, no1 = sbad[turn][4] >> 8 * half;
#pragma unroll
                for (int i = 0; i < KT * 16; ++i)
                    if ((i < 16 ? no0 : no1) >> (i % 16 / 8 * 16 + i % 8) & 1) sc[i] = __builtin_nanf("");
            }
            if (j0 < e_lo || j0 + kKeys > e_hi) {
                const int from = j0 + 8 * half - range.lo, n = range.hi - range.lo;
#pragma unroll
                for (int i = 0; i < KT * 16; ++i)
                    sc[i] = (uint32_t)(from + i / 8 * 16 + i % 8) < (uint32_t)n ? sc[i] : kNegInf;
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
        }
        if (marked && (sbad[turn][1] | sbad[turn][2]) != 0) {
            // keys with values that are not finite: what they add to the rows that see them, one key at a time, then
            // their values are cleared
            for (int half_of = 0; half_of < KT; ++half_of) {
                for (uint32_t left = uni(sbad[turn][1 + half_of]); left != 0; left &= left - 1) {
                    const int r = half_of * 32 + __ffs((int)left) - 1;
                    if (!here) continue;
                    uint32_t w = 0;
#pragma unroll
                    for (int i = 0; i < KT * 8; ++i) {
                        const uint4& x = pw[i / 4];
                        const uint32_t y = i % 4 == 0 ? x.x : i % 4 == 1 ? x.y : i % 4 == 2 ? x.z : x.w;
                        w = i == (r >> 4) * 4 + (r & 7) / 2 ? y : w;
                    }
                    float weight = __uint_as_float(r & 1 ? w & 0xffff0000u : w << 16);
                    weight = __shfl(weight, col + 32 * (r >> 3 & 1), 64);
                    const bool seen = (uint32_t)(j0 + r - range.lo) < (uint32_t)(range.hi - range.lo);
                    const char* v_at = vs + (r >> 3) * kGroup + (r & 7) * 128 + half * 8;
                    const int swap = value_swap(r) * 16;
#pragma unroll
                    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const uint2 v = *reinterpret_cast<const uint2*>(v_at + dt / 2 * 1024 + (dt % 2 * 64 ^ swap) + x * 16);
                            const float f[4] = {__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                                                __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float y = o[dt][4 * x + e];
                                o[dt][4 * x + e] = seen ? __builtin_fmaf(weight, f[e], y) : y;
                            }
                        }
                }
            }
            __syncthreads();
            for (int i = tid; i < kKeys * NI * 8; i += kThreads) {
                const int r = i / (NI * 64) * 8 + i / 8 % 8;  // 64 pieces to a block
                if (sbad[turn][1 + (r >> 5)] >> (r & 31) & 1)
                    *reinterpret_cast<uint4*>(smem + kBuf + i * 16) = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
        }
        if (here) {
#pragma unroll
            for (int i = 0; i < KT * 2; ++i)
#pragma unroll
                for (int dt = 0; dt < DT; ++dt) {
                    const char* at = vs + (v_base ^ (dt % 2 * 64)) + dt / 2 * 1024 + i * 2 * kGroup;
                    const s16x4_t a0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
                    const s16x4_t a1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 512));
                    const uint2 b0 = __builtin_bit_cast(uint2, a0), b1 = __builtin_bit_cast(uint2, a1);
                    o[dt] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(as_bf16x8(make_uint4(b0.x, b0.y, b1.x, b1.y)),
                                                                    as_bf16x8(pw[i]), o[dt], 0, 0, 0);
                }
        }
        if (more) stage(t + 1, other, next_turn);
        __syncthreads();
        turn = next_turn;
    };
    for (int t = t_from; t < t_to; t += 2) {
        work(t, smem0, smem1);
        if (t + 1 >= t_to) break;
        work(t + 1, smem1, smem0);
    }

    l += __shfl_xor(l, 32, 64);
    const float fix = __builtin_amdgcn_exp2f(-rest_c);
    if (!mine) return;
    const int64_t at = (int64_t)(tile.start + token) * p.a.Hq + qhead;
    if (p.splits > 1) {
        float* part = place(p, from_end, head, split);
        const int r = wave * 32 + col;
        if (half == 0) part[2 * r] = m, part[2 * r + 1] = l * fix;
        float* to = part + 2 * kRows + r * p.dim + half * 4;
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
    const dim3 grid(groups), block(kThreads);
    if constexpr (kHeld == BD_BF16 && kW % 64 == 0) {  // whole blocks only
        if (p.dim == kW) {
            hipLaunchKernelGGL((prompt_kernel<kW, kHeld, kForm, true>), grid, block, 0, s, p);
            return;
        }
    }
    hipLaunchKernelGGL((prompt_kernel<kW, kHeld, kForm, false>), grid, block, 0, s, p);
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
