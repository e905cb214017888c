// attend_device.h -- what the attention kernels share: the rows of a tile, query
// fragments, the running normalisation of values, partial results.
//
// Scores are kept in units of log 2: x = log2(e) * scale * q.k.  A tile's weights are
// p = 2^(x - r + 8) with r a row's reference, at most 6 below its largest score so far:
// r moves (and what is summed is rescaled) only when a score passes r + 6, which
// after the first tiles is seldom, and p stays within fp16 (2^14) with 2^-24 of
// the largest left at its end.
#pragma once

#include "kv_device.h"

namespace qmm {

constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kBias = 8.0f, kSlack = 6.0f;

// log2 of 0 and of sums in fp32
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_fast(float x) { return __builtin_amdgcn_logf(x); }

// positions [lo, hi) of the keys that row i (of count, length len) sees
__device__ __forceinline__ void attend_span(const AttendArgs &a, const KvRows &rows, int i, int &lo, int &hi) {
    const int pos = rows.len - rows.count + i;
    hi = a.causal ? pos + 1 : rows.len;
    hi = hi > rows.len ? rows.len : hi;
    lo = a.window > 0 && pos + 1 > a.window ? pos + 1 - a.window : 0;
}

// 2^e as a float, |e| <= 126
__device__ __forceinline__ float pow2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// A query row's power of two: its largest magnitude's exponent becomes 12, so that fp16
// pieces of it keep what fp32 holds (two) or the type itself (one), down to 2^-24 of
// the row's largest.  `top`: the largest |q| bits of the row (an infinity or NaN: 255).
__device__ __forceinline__ int query_shift(uint32_t top) {
    const int e = (int)(top >> 23) - 127;  // zero and subnormals: -127
    return e < -114 ? 126 : 12 - e;
}

// elements of a word as key_codes holds them: 0 4 1 5 2 6 3 7, the odd ones over 16, which
// the codes' places take back
template <int PIECES>
__device__ __forceinline__ void query_pieces(const float *x, float by, h8 &hi, h8 &lo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = x[(i >> 1) + 4 * (i & 1)] * ((i >> 1) & 1 ? by * 0.0625f : by);
        hi[i] = (_Float16)v;
        if constexpr (PIECES == 2) lo[i] = (_Float16)(v - (float)hi[i]);
    }
}

// Constants of the decode in registers: an instruction of this family takes no
// literals, and one scalar register at most.
struct Decode {
    uint32_t low, high;  // 0x000f000f, 0x00f000f0 (scalar)
    uint32_t magic;      // 1024 in both halves (vector)
    __device__ __forceinline__ void set() {
        asm("s_mov_b32 %0, 0x000f000f" : "=s"(low));
        asm("s_mov_b32 %0, 0x00f000f0" : "=s"(high));
        asm("v_mov_b32 %0, 0x64006400" : "=v"(magic));
    }
    // 1024 + u of the codes in bits 0..3 of both halves; 1024 + 16 u of those in bits 4..7
    __device__ __forceinline__ h2 even(uint32_t x) const { return as_h2((x & low) | magic); }
    __device__ __forceinline__ h2 odd(uint32_t x) const { return as_h2((x & high) | magic); }
};
// u - 8 and 16 (u - 8), exact
__device__ __forceinline__ h2 centred_even(h2 x) { return x - h2{(_Float16)1032.0f, (_Float16)1032.0f}; }
__device__ __forceinline__ h2 centred_odd(h2 x) { return x - h2{(_Float16)1152.0f, (_Float16)1152.0f}; }

// eight codes of a word against query_pieces
__device__ __forceinline__ h8 key_codes(const Decode &k, uint32_t w) {
    const h2 a = centred_even(k.even(w)), b = centred_odd(k.odd(w)), c = centred_even(k.even(w >> 8)),
             d = centred_odd(k.odd(w >> 8));
    return h8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// max over the wavefront of two 16-bit values per lane
__device__ __forceinline__ uint32_t wave_max_u16x2(uint32_t v) {
    uint32_t m = (v & 0xffffu) > (v >> 16) ? v & 0xffffu : v >> 16;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint32_t u = __shfl_xor(m, o, 64);
        m = u > m ? u : m;
    }
    return m;
}
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// The power of two that value scales are multiplied by, from the largest scale's bits:
// its exponent becomes 7 (products with codes, 16-fold ones too, stay within fp16; a scale below
// 2^-21 of the largest is rounded to a step of 2^-31 of it); at most 2^15.
__device__ __forceinline__ int value_shift(uint32_t top) {
    const int e = (int)(top >> 10);
    return e < 7 ? 15 : 22 - e;
}

typedef float f16v __attribute__((ext_vector_type(16)));
__device__ __forceinline__ f4 mfma16(h8 a, h8 b, f4 c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
__device__ __forceinline__ f16v mfma32(h8 a, h8 b, f16v c) { return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0); }

// ---- who takes a sequence, and where its splits' parts go.  Query rows of a sequence
// and cache head: token * group + head of the group.  Up to few_room of them (all, where
// every sequence has one token) go to attention.hip's kernel in tiles of kFewTile, more to
// attend_rows.hip's in tiles of kManyTile.
constexpr int kFewTile = 16, kManyTile = 256;
// The most rows whose entries' weights k_attend_mass forms, which converts the queries anew for every 32 entries;
// attend_mass.hip's kernel has the more, from queries that the attention left.  What the weights add to a call, us, here and
// there, 16 sequences of 4000 entries, 8 heads of 128: bf16 of 32 rows 50 and 59, 48: 60 and 61, 64: 72 and 60, 256: 201 and
// 99; fp32 32: 57 and 82, 48: 73 and 86, 64: 87 and 85, 512: 487 and 248; heads of 64 in bf16 32: 27 and 45, 64: 38 and 47;
// of 256, whose rows do not stay in registers here, 4: 110 and 95, 64: 262 and 99.
constexpr int kMassRoom = 32;

struct Splits {
    int few_room;
    int few_tiles, many_tiles;  // tiles at most (starts that do not ascend could say more)
    int few_want, many_want;    // workgroups of a cache head that fill the GPU
    int few_most, many_most;    // splits at most
    int few_rows;             // rows of a tile that can have any (many: kManyTile)
    float *few_sums;          // [split][tile][head][few_rows][D]
    float2 *few_stats;        // [split][tile][head][few_rows]: (reference - bias, sum)
    float *many_sums;         // the same, of kManyTile rows
    float2 *many_stats;
    // for the weights of the entries, by (cache head, token, head of the group): attend_group_row
    float *lse2;              // [heads * T * group] in log2 units, or null
    // and what sequences of more than kMassRoom rows leave for attend_mass.hip, or null:
    _Float16 *queries;        // [pieces][heads * T * group][D], as query_pieces has them
    int64_t query_piece;      // elements of a piece
    float *factors;           // [heads * T * group], of the rows' products
};

// The tiles of a call that have rows of one of the two kernels, in the sequences' order, and into how many splits
// of the entries each goes: the GPU's workgroups over the tiles.  Only the device knows how many rows a sequence has,
// so each wavefront counts them: sequence 64 k + lane's tiles end at upto[k].  All tiles of a call go into as many
// splits, whatever their sequences' lengths: one of 131072 entries takes 51 us alone, and among 63 of 500, where the tiles
// fill the GPU and nothing is split, 1308 (fp32, 8 heads of 128).  Beyond kCounted sequences counting takes too long;
// there sequence b's tiles start at slot floor(starts[b] * group / ROWS) + b, not all slots have rows, and nothing is
// split either.
constexpr int kCounted = 256;
// sum over the lanes up to this one
__device__ __forceinline__ int wave_upto(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // the lane 1, 2, 4, 8 below, in rows of 16
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row 0's last lane to row 1, 2's to 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row 1's last lane to rows 2 and 3
    return v;
}
template <int ROWS>
struct Tiles {
    int upto[kCounted / 64], own[kCounted / 64];
    KvRows rows[kCounted / 64];
    int live, splits;

    __device__ __forceinline__ void open(const AttendArgs &a, const Splits &sp) {
        constexpr bool many = ROWS == kManyTile;
        const int room = sp.few_room, want = many ? sp.many_want : sp.few_want, most = many ? sp.many_most : sp.few_most;
        const int lane = threadIdx.x & 63;
        splits = 1;
        if (a.c.starts == nullptr) live = a.c.B * ((a.group + ROWS - 1) / ROWS);
        else if (a.c.B > kCounted) {
            live = a.c.T * a.group / ROWS + a.c.B;
            return;
        } else {
            live = 0;
#pragma unroll
            for (int k = 0; k < kCounted / 64; ++k) {
                if (64 * k >= a.c.B) break;
                const int b = 64 * k + lane;
                rows[k] = kv_rows(a.c, b < a.c.B ? b : a.c.B - 1);
                const int n = b < a.c.B ? rows[k].count * a.group : 0;
                own[k] = (n > room) == many ? (n + ROWS - 1) / ROWS : 0;
                upto[k] = live + wave_upto(own[k]);
                live = __builtin_amdgcn_readlane(upto[k], 63);
            }
            const int tiles = many ? sp.many_tiles : sp.few_tiles;
            live = live < tiles ? live : tiles;
        }
        if (live > 0) {
            const int n = want / live;
            splits = n > most ? most : (n < 1 ? 1 : n);
        }
    }
    // the sequence, its rows and tile, or false (a slot without rows)
    __device__ __forceinline__ bool place(const AttendArgs &a, int at, int &b, int &tile, KvRows &its) const {
        if (a.c.starts == nullptr) {
            const int per = (a.group + ROWS - 1) / ROWS;
            b = at / per;
            tile = at - b * per;
            its = kv_rows(a.c, b);
            return true;
        }
        if (a.c.B > kCounted) {
            auto slot = [&](int i) {
                const int t = a.c.starts[i];
                return (int64_t)(t < 0 ? 0 : (t > a.c.T ? a.c.T : t)) * a.group / ROWS + i;
            };
            b = __builtin_amdgcn_readfirstlane(kv_last_not_above(a.c.B, at, slot));
            if (b < 0) return false;
            tile = __builtin_amdgcn_readfirstlane((int)(at - slot(b)));
            its = kv_rows(a.c, b);
            return tile >= 0;  // below 0: starts that do not ascend
        }
#pragma unroll
        for (int k = 0; k < kCounted / 64; ++k) {
            if (64 * k >= a.c.B) break;
            const uint64_t past = __ballot(upto[k] > at);
            if (past == 0) continue;
            const int l = __builtin_ctzll(past);
            b = 64 * k + l;
            tile = at - __builtin_amdgcn_readlane(upto[k] - own[k], l);
            its.first = __builtin_amdgcn_readlane(rows[k].first, l);
            its.count = __builtin_amdgcn_readlane(rows[k].count, l);
            its.len = __builtin_amdgcn_readlane(rows[k].len, l);
            return true;
        }
        return false;
    }
};

// the row of the batch's output, token * query heads + head, of a sequence's query row
__device__ __forceinline__ int64_t attend_out_row(const AttendArgs &a, const KvRows &rows, int head, int row) {
    const int token = row / a.group, h = row - token * a.group;
    return (int64_t)(rows.first + token) * (a.c.heads * a.group) + head * a.group + h;
}
// where an output row starts in q or out
__device__ __forceinline__ int64_t attend_at(const AttendArgs &a, int64_t out_row, int64_t ld) {
    const int heads = a.c.heads * a.group;
    const int64_t token = out_row / heads;
    return token * ld + (out_row - token * heads) * a.c.D;
}
// four elements of an output row
__device__ __forceinline__ void attend_store4(int type, void *out, int64_t at, float a, float b, float c, float d) {
    if (type == 0) *reinterpret_cast<float4 *>(static_cast<float *>(out) + at) = make_float4(a, b, c, d);
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(out) + at) =
            type == 1 ? make_uint2(f32_to_f16_bits(a) | f32_to_f16_bits(b) << 16, f32_to_f16_bits(c) | f32_to_f16_bits(d) << 16)
                      : make_uint2(bf16_bits(a) | bf16_bits(b) << 16, bf16_bits(c) | bf16_bits(d) << 16);
}
// the place of a token's query head among the rows of its cache head
__device__ __forceinline__ int64_t attend_group_row(const AttendArgs &a, int token, int head, int of_group) {
    return ((int64_t)head * a.c.T + token) * a.group + of_group;
}
__device__ __forceinline__ void attend_lse(const AttendArgs &a, float *lse2, int64_t out_row, float l2) {
    if (a.lse != nullptr) a.lse[out_row] = l2 * kLn2;
    if (lse2 == nullptr) return;
    const int row = (int)out_row, token = row / (a.c.heads * a.group), q_head = row - token * (a.c.heads * a.group);
    const int head = q_head / a.group;
    lse2[attend_group_row(a, token, head, q_head - head * a.group)] = l2;
}

// attend_rows.hip: sequences of more than few_room rows; whether it has a kernel for such rows
constexpr bool attend_rows_has(int type, int64_t D) { return D <= (type == 0 ? 128 : 192); }
hipError_t launch_attend_rows(int type, const AttendArgs &a, const Splits &sp, int64_t workgroups, hipStream_t s);

// attend_mass.hip: the weights of their entries
hipError_t launch_attend_mass_rows(int type, const AttendArgs &a, const Splits &sp, hipStream_t s);

}  // namespace qmm
