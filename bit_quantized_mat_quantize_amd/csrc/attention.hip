// attention.hip -- attention over the paged 4-bit cache, few rows per sequence
// (gfx950): one token, or some, of each sequence against all its entries; the joint of
// splits; and the weights that entries get from few rows.
//
// A workgroup takes one tile of 16 query rows (row = token * group + head of the
// group, so that one read of an entry serves the whole group), one cache head and
// one split of the entries; its four wavefronts take 32 entries each in turn, by direct
// loads into rings of LDS of their own, a step ahead, and are joined at the end.  Per 32
// entries:
//
//   S^T = K Q^T     16 entries x 16 rows per matrix instruction, one per block of 32
//                   elements: the codes are exact in fp16, the block's scale multiplies
//                   the fp32 result.  fp32 queries are two fp16 pieces (22 bits).
//   O^T += V^T P^T  a lane holds eight entries' words of the same eight elements, so the
//                   codes are transposed by byte permutes within the lane; code * scale
//                   is rounded to fp16 for 16-bit queries, and cut in two exact pieces for
//                   fp32 ones.  p is rounded to fp16 for bf16 queries, and two pieces for fp16
//                   and fp32 ones: rounded to one it put fp16 outputs on short contexts at up to
//                   1.6 times the 64-bit error that fp16 itself costs (1.4 with two; of 40 random
//                   calls), and two are a twentieth of the time (32 sequences of 8192
//                   entries, 8 query heads of a cache head of 128: 70 us and 74; with 256
//                   rows, 16 of 4000: 193 and 211).
//
// In both products the entries lie along the registers of a lane and the rows along
// the lanes, so softmax needs no exchange between lanes, and P goes from one product
// to the next as it is.
//
// An entry whose page is not in the pool, or that has a NaN scale, makes the rows that
// see it NaN: its score becomes NaN and its values 0, so that rows that do not see it
// are not touched.
//
// Bounds: single tokens of long contexts, the issue of vector instructions beside the
// bytes (56% of the issue slots and matrix instructions 21% of the cycles for fp32 queries,
// 51% and 10% for 16-bit ones; 32 sequences of up to 8192 entries, 8 cache heads of 128, fp32: 66 us,
// 3.8 TB/s of the cache; 2 of 131072 in bf16: 61 us, 4.5 TB/s); many rows, the same once per 16 of them;
// one short sequence, a chain of latencies (8 us for 1000 entries).
#include "attend_device.h"

namespace qmm {
namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kRows = kFewTile;  // query rows of a tile
constexpr int kKeys = 32;  // entries of a wavefront's step

// What a lane reads of 32 entries.  Lane (n, g), n = lane & 15, g = lane >> 4:
//   k[s]  words (b, g) of all blocks b of entry 16 s + n
//   v[s]  words n (and 16 + n for D > 128) of the entries 16 s + 4 g .. + 3
//   ks[s] the key scales of these four entries, block by block; vs[s] the value scales of
//         the blocks that hold word n (and 16 + n)
template <int D>
struct Step {
    static constexpr int NB = D / 32, ROUNDS = D > 128 ? 2 : 1;
    uint32_t k[2][NB];
    uint4 v[2][ROUNDS];
    uint2 ks[2][NB], vs[2][ROUNDS];
    int bad;  // bit s: entries 16 s .. 16 s + 15 have no page
};

template <int D>
__device__ __forceinline__ void read_step(const KvCache &c, int b, int head, int k0, int last, Step<D> &t) {
    constexpr int NB = Step<D>::NB, ROUNDS = Step<D>::ROUNDS, WORDS = D / 8;
    const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
    t.bad = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        int at = k0 + 16 * s;
        at = at > last ? last : at;  // the last 16 entries that hold anything
        int page = kv_page(c, b, at);
        if (page < 0) t.bad |= 1 << s;
        page = page < 0 ? 0 : page;
        const uint8_t *kc = kv_chunk(c, page, 0, head), *vc = kv_chunk(c, page, 1, head);
        const int e0 = at & ((1 << c.page_log2) - 1);
        const uint32_t *kw = reinterpret_cast<const uint32_t *>(kc) + (e0 + n) * WORDS + g * NB;
        if constexpr (NB % 4 == 0) {
#pragma unroll
            for (int i = 0; i < NB / 4; ++i) {
                const uint4 u = ld16(kw + 4 * i);
                t.k[s][4 * i] = u.x, t.k[s][4 * i + 1] = u.y, t.k[s][4 * i + 2] = u.z, t.k[s][4 * i + 3] = u.w;
            }
        } else if constexpr (NB % 2 == 0) {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) {
                const uint2 u = *reinterpret_cast<const uint2 *>(kw + 2 * i);
                t.k[s][2 * i] = u.x, t.k[s][2 * i + 1] = u.y;
            }
        } else {
#pragma unroll
            for (int i = 0; i < NB; ++i) t.k[s][i] = kw[i];
        }
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const int w = (16 * r + n) % WORDS;
            t.v[s][r] = ld16(reinterpret_cast<const uint32_t *>(vc) + kv_value_word(D, e0 + 4 * g, w));
            t.vs[s][r] = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(vc) + kv_scale_at(c, e0 + 4 * g, w >> 2));
        }
#pragma unroll
        for (int i = 0; i < NB; ++i)
            t.ks[s][i] = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(kc) + kv_scale_at(c, e0 + 4 * g, i));
    }
}

// A lane's share of 16 query rows: row n, elements 8 g .. 8 g + 7 of each block
template <int PIECES, int D>
struct Query {
    h8 hi[D / 32], lo[PIECES == 2 ? D / 32 : 1];

    __device__ __forceinline__ void set(const float (&x)[D / 32][8], float by) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) query_pieces<PIECES>(x[i], by, hi[i], lo[PIECES == 2 ? i : 0]);
    }
};

// Products of 32 entries with the queries: x[4 s + r] is entry 16 s + 4 g + r against row n.
template <int PIECES, int D>
__device__ __forceinline__ void products(const Decode &k, const Step<D> &t, const Query<PIECES, D> &q, float *x) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        f4 acc = {0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            const h8 codes = key_codes(k, t.k[s][b]);
            f4 dot = mfma16(codes, q.hi[b], f4{0, 0, 0, 0});
            if constexpr (PIECES == 2) dot = mfma16(codes, q.lo[b], dot);
            const h2 d0 = as_h2(t.ks[s][b].x), d1 = as_h2(t.ks[s][b].y);
            acc[0] = fmaf((float)d0.x, dot[0], acc[0]);
            acc[1] = fmaf((float)d0.y, dot[1], acc[1]);
            acc[2] = fmaf((float)d1.x, dot[2], acc[2]);
            acc[3] = fmaf((float)d1.y, dot[3], acc[3]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * s + r] = acc[r];
    }
    if (__builtin_expect(t.bad != 0, 0)) {  // the same for the whole wavefront
        asm volatile("");                      // not worth eight selects in every step
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (t.bad >> (i >> 2)) & 1 ? __builtin_nanf("") : x[i];
    }
}

// workgroups that a CU holds, by their registers
template <int PIECES, int D>
constexpr int at_once = D > 128 ? 2 : (PIECES == 2 && D == 128 ? 3 : 4);

// ---- a wavefront's ring of steps in LDS, filled by direct loads.  16 entries of a head are
// one run of D/2 * 16 bytes of codes, for keys and for values alike, so a lane's place
// in a load is fixed and only its page's base and the entry's offset, both scalar, change.
// A group's image: keys' codes, values' codes, filler to 1 KiB; scales as [keys or
// values][block][16 entries], filler to 256 bytes.
template <int D>
struct Ring {
    static constexpr int CODES = (16 * D + 1023) / 1024, SCALES = (2 * D + 255) / 256;  // load instructions
    static constexpr int SCALE_AT = 1024 * CODES, GROUP = SCALE_AT + 256 * SCALES, BYTES = 2 * GROUP;
    static constexpr int LOADS = 2 * (CODES + SCALES);
    static constexpr int SLOTS = 2;  // steps in LDS
    static constexpr int WAVE = SLOTS * BYTES;
    uint32_t code_at[CODES], scale_at[SCALES];  // this lane's place in a chunk pair, per instruction
    uint32_t records;                           // bytes from a page's keys to the end of its values, of one head
    uint32_t lds;                               // this wavefront's ring
    const uint8_t *ring;

    __device__ __forceinline__ void set(const KvCache &c, const uint8_t *mine) {
        const int lane = threadIdx.x & 63;
        const uint32_t chunk = (uint32_t)kv_chunk_bytes(c), values = chunk * (uint32_t)c.heads;
#pragma unroll
        for (int i = 0; i < CODES; ++i) {
            int p = 64 * i + lane;  // 16-byte piece of keys, then of values
            p = p < D ? p : D - 1;
            code_at[i] = p < D / 2 ? p * 16 : values + (p - D / 2) * 16;
        }
#pragma unroll
        for (int i = 0; i < SCALES; ++i) {
            int p = 64 * i + lane;  // 4-byte piece
            p = p < D / 2 ? p : D / 2 - 1;
            const int part = p / (D / 4), b = p % (D / 4) / 8, e = p % 8;
            scale_at[i] = part * values + (((D / 2) << c.page_log2) + 2 * (b << c.page_log2)) + 4 * e;
        }
        records = values + chunk;
        ring = mine;
        lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t *)mine);
    }
    // 16 entries from entry e0 of a page on (base: its keys) into half s of a slot
    __device__ __forceinline__ void load(int slot, int s, const uint8_t *base, int e0) const {
        const uint64_t at = (uint64_t)(uintptr_t)base;
        const u32x4 r = {(uint32_t)at, (uint32_t)(at >> 32) & 0xffffu, records, 0x00020000u};
        const uint32_t to = lds + slot * BYTES + s * GROUP;
#pragma unroll
        for (int i = 0; i < CODES; ++i)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to + 1024 * i),
                         "v"(code_at[i]), "s"(r), "s"(e0 * (D / 2)) : "m0", "memory");
#pragma unroll
        for (int i = 0; i < SCALES; ++i)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(to + SCALE_AT + 256 * i),
                         "v"(scale_at[i]), "s"(r), "s"(e0 * 2) : "m0", "memory");
    }
    __device__ __forceinline__ void read(int slot, Step<D> &t) const {
        constexpr int NB = D / 32, ROUNDS = Step<D>::ROUNDS, WORDS = D / 8;
        const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const uint8_t *from = ring + slot * BYTES + s * GROUP;
            const uint32_t *kw = reinterpret_cast<const uint32_t *>(from) + n * WORDS + g * NB;
            if constexpr (NB % 4 == 0) {
#pragma unroll
                for (int i = 0; i < NB / 4; ++i) {
                    const uint4 u = ld16(kw + 4 * i);
                    t.k[s][4 * i] = u.x, t.k[s][4 * i + 1] = u.y, t.k[s][4 * i + 2] = u.z, t.k[s][4 * i + 3] = u.w;
                }
            } else if constexpr (NB % 2 == 0) {
#pragma unroll
                for (int i = 0; i < NB / 2; ++i) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(kw + 2 * i);
                    t.k[s][2 * i] = u.x, t.k[s][2 * i + 1] = u.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) t.k[s][i] = kw[i];
            }
            const uint8_t *sc = from + SCALE_AT + 8 * g;
#pragma unroll
            for (int i = 0; i < NB; ++i) t.ks[s][i] = *reinterpret_cast<const uint2 *>(sc + 32 * i);
#pragma unroll
            for (int r = 0; r < ROUNDS; ++r) {
                const int w = (16 * r + n) % WORDS;
                t.v[s][r] = ld16(from + 8 * D + (g * WORDS + w) * 16);
                t.vs[s][r] = *reinterpret_cast<const uint2 *>(sc + 32 * (NB + (w >> 2)));
            }
        }
    }
};

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
// until at most n steps' loads are on their way (0 <= n < SLOTS, the same for the wavefront)
template <int LOADS, int MOST>
__device__ __forceinline__ void wait_steps(int n) {
    if constexpr (MOST > 0) {
        if (n >= MOST) {
            wait_loads<MOST * LOADS>();
            return;
        }
        wait_steps<LOADS, MOST - 1>(n);
    } else wait_loads<0>();
}

// A tile's rows and the queries of this lane's row
template <int PIECES, int D>
struct Tile {
    KvRows rows;
    int b, row;        // sequence; this lane's row of it, token * group + head
    bool live;         // the row exists
    int lo, hi;        // entries that it sees
    int first, last;   // entries that any row of the tile sees: [first, last)
    int all_lo, all_hi;  // entries that every row sees
    float factor;      // of the dot products of codes, to log2 units
    int batch_row, q_head;
    Query<PIECES, D> q;

    // what the rows see; their queries come later, so that entries can be on their way first
    __device__ __forceinline__ bool open(const AttendArgs &a, int seq, const KvRows &its, int tile, int head) {
        b = seq;
        rows = its;
        const int lane = threadIdx.x & 63, n = lane & 15, total = rows.count * a.group;
        const int r0 = tile * kRows;
        if (r0 >= total) return false;
        const int r1 = r0 + kRows - 1 < total ? r0 + kRows - 1 : total - 1;
        row = r0 + n;
        live = row < total;
        const int use = live ? row : r1, token = use / a.group;
        attend_span(a, rows, token, lo, hi);
        attend_span(a, rows, r0 / a.group, first, all_hi);
        attend_span(a, rows, r1 / a.group, all_lo, last);
        batch_row = rows.first + token;
        q_head = head * a.group + use - token * a.group;
        return true;
    }
    // the row in lse, and where it starts in q or out
    __device__ __forceinline__ int64_t out_row(const AttendArgs &a) const {
        return (int64_t)batch_row * (a.c.heads * a.group) + q_head;
    }
    __device__ __forceinline__ int64_t at_row(int64_t ld) const { return batch_row * ld + (int64_t)q_head * D; }
    __device__ __forceinline__ void queries(const AttendArgs &a) {
        const int64_t at = at_row(a.ld_q) + 8 * ((threadIdx.x & 63) >> 4);
        float x[D / 32][8];
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            kv_load8(type, a.q, at + 32 * i, x[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(x[i][j]) & 0x7fffffffu;
                top = u > top ? u : top;
            }
        }
        for (int o = 16; o < 64; o <<= 1) {
            const uint32_t u = __shfl_xor(top, o, 64);
            top = u > top ? u : top;
        }
        const int shift = query_shift(top);
        q.set(x, a.scale < 0.0f ? -pow2i(shift) : pow2i(shift));
        factor = (top >> 23) == 255 ? __builtin_nanf("") : fabsf(a.scale) * pow2i(-shift);
    }
    int type;
};

// One wavefront's running result: row n, elements 8 w + j at sums[r][w's round][j] ...
template <int D>
struct Running {
    static constexpr int ROUNDS = Step<D>::ROUNDS;
    f4 o[ROUNDS][8];   // o[round][j][r]: element 8 * (16 * round + 4 g + r) + j
    float ref, sum;    // the row's reference; this lane's part of the sum of p
    uint32_t bound;    // value scales up to these bits need no other power of two
    int shift;         // o holds sums times 2^shift

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) o[r][j] = f4{0, 0, 0, 0};
        ref = -INFINITY;
        sum = 0.0f;
        bound = 0;
        shift = 15;
    }
    __device__ __forceinline__ void scale(float by) {
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) o[r][j] *= by;
    }
};

// WP: pieces of a weight.  masked: some row does not see some entry of the step
template <int PIECES, int WP, int D>
__device__ __forceinline__ void step(const Decode &k, Step<D> &t, const Tile<PIECES, D> &q, int k0, bool masked, Running<D> &run) {
    constexpr int ROUNDS = Step<D>::ROUNDS;
    const int lane = threadIdx.x & 63, g = lane >> 4;
    float x[8];
    products<PIECES, D>(k, t, q.q, x);
    if (masked) {  // entries that no row sees hold anything
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = k0 + 16 * s + 4 * g + 2 * i;
                const uint32_t keep = (at >= q.first && at < q.last ? 0xffffu : 0u) |
                                      (at + 1 >= q.first && at + 1 < q.last ? 0xffff0000u : 0u);
#pragma unroll
                for (int r = 0; r < ROUNDS; ++r) (i ? t.vs[s][r].y : t.vs[s][r].x) &= keep;
            }
    }
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
            top = max_u16x2(top, max_u16x2(t.vs[s][r].x & 0x7fff7fffu, t.vs[s][r].y & 0x7fff7fffu));
    if (__any((top & 0xffffu) >= run.bound || (top >> 16) >= run.bound)) {
        // a scale beyond all so far, or one that is not finite
        if (wave_max_u16x2(top) >= 0x7c00u) {
            uint32_t bad = 0;  // bit 4 s + r: entry 16 s + 4 g + r
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < ROUNDS; ++r) {
                    uint32_t *u[2] = {&t.vs[s][r].x, &t.vs[s][r].y};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if ((*u[i] & 0x7c00u) == 0x7c00u) bad |= 1u << (4 * s + 2 * i), *u[i] &= 0xffff0000u;
                        if ((*u[i] & 0x7c000000u) == 0x7c000000u) bad |= 2u << (4 * s + 2 * i), *u[i] &= 0xffffu;
                    }
                }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) bad |= __shfl_xor(bad, o, 64);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((bad >> i) & 1) x[i] = __builtin_nanf("");
            top = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int r = 0; r < ROUNDS; ++r)
                    top = max_u16x2(top, max_u16x2(t.vs[s][r].x & 0x7fff7fffu, t.vs[s][r].y & 0x7fff7fffu));
        }
        const uint32_t most = wave_max_u16x2(top);
        if (most >= run.bound) {
            const int shift = value_shift(most);
            run.scale(pow2i(shift - run.shift));
            run.shift = shift;
            run.bound = ((most >> 10) + 1) << 10;
        }
    }
    if (masked) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = k0 + 16 * (i >> 2) + 4 * g + (i & 3);
            x[i] *= q.factor;
            if (at < q.lo || at >= q.hi) x[i] = -INFINITY;
        }
    }
    const float factor = masked ? 1.0f : q.factor;  // x[i] * factor: scores
    float most = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7]))) * factor;
    if (__any(most > run.ref + kSlack)) {
        for (int o = 16; o < 64; o <<= 1) most = fmaxf(most, __shfl_xor(most, o, 64));
        const float ref = fmaxf(run.ref, most), by = ref == -INFINITY ? 1.0f : exp2_fast(run.ref - ref);
        run.scale(by);
        run.sum *= by;
        run.ref = ref;
    }
    const float from = run.ref == -INFINITY ? 0.0f : run.ref - kBias;
    h8 ph, pl;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float p = exp2_fast(fmaf(x[i], factor, -from));
        run.sum += p;
        ph[i] = (_Float16)p;
        if constexpr (WP == 2) pl[i] = (_Float16)(p - (float)ph[i]);
    }
    const _Float16 unit = (_Float16)pow2i(run.shift);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t w[8] = {t.v[0][r].x, t.v[0][r].y, t.v[0][r].z, t.v[0][r].w,
                               t.v[1][r].x, t.v[1][r].y, t.v[1][r].z, t.v[1][r].w};
        const uint32_t su[4] = {t.vs[0][r].x, t.vs[0][r].y, t.vs[1][r].x, t.vs[1][r].y};
        h2 d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = as_h2(su[i]) * h2{unit, unit};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            h2 code[2][4];  // elements 2y and 2y + 1 of the word (these 16-fold), entries in pairs
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t both = __builtin_amdgcn_perm(w[2 * i + 1], w[2 * i], 0x0c040c00u + 0x00010001u * y);
                code[0][i] = centred_even(k.even(both));
                code[1][i] = centred_odd(k.odd(both));
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                h8 vh, vl;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const h2 h = code[o][i] * d[i];
                    vh[2 * i] = h.x, vh[2 * i + 1] = h.y;
                    if constexpr (PIECES == 2) {
                        const h2 l = __builtin_elementwise_fma(code[o][i], d[i], -h);
                        vl[2 * i] = l.x, vl[2 * i + 1] = l.y;
                    }
                }
                f4 &acc = run.o[r][2 * y + o];
                acc = mfma16(vh, ph, acc);
                if constexpr (WP == 2) acc = mfma16(vh, pl, acc);
                if constexpr (PIECES == 2) acc = mfma16(vl, ph, acc);
            }
        }
    }
}

template <int PIECES, int WP, int D>
__global__ __launch_bounds__(kThreads, (at_once<PIECES, D>)) void k_attend(AttendArgs a, Splits sp, int type) {
    constexpr int ROUNDS = Step<D>::ROUNDS, PITCH = D + 4;
    using R = Ring<D>;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    static_assert(kWaves * R::WAVE >= 2 * kRows * PITCH * 4, "the joint of the wavefronts takes the rings' place");
    float(*buf)[kRows][PITCH] = reinterpret_cast<float(*)[kRows][PITCH]>(lds);
    __shared__ float2 stats[kWaves][kRows];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int head = blockIdx.x % a.c.heads, x = blockIdx.x / a.c.heads;
    Tiles<kRows> tiles;
    tiles.open(a, sp);
    const int splits = tiles.splits, place = x / splits, split = x - place * splits;
    int b, tile;
    KvRows rows;
    if (place >= tiles.live || !tiles.place(a, place, b, tile, rows)) return;
    if (rows.count * a.group > sp.few_room) return;  // the other kernel's
    Tile<PIECES, D> q;
    q.type = type;
    if (!q.open(a, b, rows, tile, head)) return;
    q.queries(a);
    if (sp.queries != nullptr && split == 0 && wave == 0 && q.live && rows.count * a.group > kMassRoom) {
        const int64_t row = attend_group_row(a, rows.first, head, q.row);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            _Float16 *p = sp.queries + row * D + 32 * i + 8 * g;
            *reinterpret_cast<h8 *>(p) = q.q.hi[i];
            if constexpr (PIECES == 2) *reinterpret_cast<h8 *>(p + sp.query_piece) = q.q.lo[i];
        }
        if (g == 0) sp.factors[row] = q.factor;
    }
    Running<D> run;
    run.clear();
    // this split's steps of 32 entries: whole rounds of the four wavefronts
    const int s0 = (q.first < 0 ? 0 : q.first) / kKeys, s1 = q.last > 0 ? (q.last + kKeys - 1) / kKeys : 0;
    const int rounds = s1 > s0 ? (s1 - s0 + kWaves - 1) / kWaves : 0;
    const int from = s0 + (int)((int64_t)rounds * split / splits) * kWaves;
    const int to0 = s0 + (int)((int64_t)rounds * (split + 1) / splits) * kWaves;
    const int to = to0 < s1 ? to0 : s1, last16 = q.last > 0 ? (q.last - 1) & ~15 : 0;
    const int at0 = __builtin_amdgcn_readfirstlane(from + wave), steps = __builtin_amdgcn_readfirstlane(at0 < to ? (to - at0 + kWaves - 1) / kWaves : 0);
    if (steps > 0) {
        R ring;
        ring.set(a.c, lds + wave * R::WAVE);
        Decode decode;
        decode.set();
        typedef const __attribute__((address_space(4))) int32_t *scalar_ints;
        const scalar_ints table = (scalar_ints)(uintptr_t)(a.c.table + (int64_t)b * a.c.width);
        uint32_t bad = 0;  // of the steps on their way, two bits each, the next one lowest
        auto issue = [&](int i) {
            const int k0 = (at0 + i * kWaves) * kKeys, slot = i % R::SLOTS;
            uint32_t none = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int at = k0 + 16 * s < last16 ? k0 + 16 * s : last16;  // the last 16 entries that hold anything
                int page = table[at >> a.c.page_log2];
                if (page < 0 || page >= a.c.pages) {
                    none |= 1u << s;
                    page = 0;
                }
                ring.load(slot, s, kv_chunk(a.c, page, 0, head), at & ((1 << a.c.page_log2) - 1));
            }
            bad |= none << (2 * ((R::SLOTS - 1)));
        };
        constexpr int AHEAD = R::SLOTS - 1;
        for (int i = 0; i < AHEAD; ++i) {
            bad >>= 2;
            if (i < steps) issue(i);
        }
        for (int i = 0; i < steps; ++i) {
            bad >>= 2;
            if (i + AHEAD < steps) issue(i + AHEAD);
            const int later = steps - 1 - i < AHEAD ? steps - 1 - i : AHEAD;
            wait_steps<R::LOADS, AHEAD>(later);
            Step<D> t;
            ring.read(i % R::SLOTS, t);
            t.bad = bad & 3;
            const int k0 = (at0 + i * kWaves) * kKeys;
            step<PIECES, WP, D>(decode, t, q, k0, k0 < q.all_lo || k0 + kKeys > q.all_hi, run);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // this slot's reads are done
        }
    }
    __syncthreads();  // the rings' place is the joint's now
    for (int o = 16; o < 64; o <<= 1) run.sum += __shfl_xor(run.sum, o, 64);
    // the wavefronts' parts, to the largest reference
    if (g == 0) stats[wave][n] = make_float2(run.ref, run.sum);
    __syncthreads();
    float ref = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) ref = fmaxf(ref, stats[w][n].x);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const float2 s = stats[w][n];
        sum += s.x == -INFINITY ? s.y : s.y * exp2_fast(s.x - ref);  // a NaN stands in sums without a reference too
    }
    const float by = (run.ref == -INFINITY ? 1.0f : exp2_fast(run.ref - ref)) * pow2i(-run.shift);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
        for (int j = 1; j < 8; j += 2) run.o[r][j] *= 0.0625f;  // the odd elements' codes were 16-fold
    for (int half = 2; half >= 1; half >>= 1) {  // wavefronts half .. 2 half - 1 into 0 .. half - 1
        if (wave >= half && wave < 2 * half) {
#pragma unroll
            for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int w = 16 * r + 4 * g + i;
                    if (w < D / 8) {
                        float4 *o = reinterpret_cast<float4 *>(&buf[wave - half][n][8 * w]);
                        const float f = half == 2 || wave != 1 ? by : 1.0f;
                        o[0] = make_float4(run.o[r][0][i] * f, run.o[r][1][i] * f, run.o[r][2][i] * f, run.o[r][3][i] * f);
                        o[1] = make_float4(run.o[r][4][i] * f, run.o[r][5][i] * f, run.o[r][6][i] * f, run.o[r][7][i] * f);
                    }
                }
        }
        __syncthreads();
        if (wave < half) {
#pragma unroll
            for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int w = 16 * r + 4 * g + i;
                    if (w < D / 8) {
                        const float *o = &buf[wave][n][8 * w];
#pragma unroll
                        for (int j = 0; j < 8; ++j) run.o[r][j][i] = run.o[r][j][i] * (half == 2 ? by : 1.0f) + o[j];
                    }
                }
        }
        __syncthreads();
    }
    if (wave != 0 || !q.live) return;
    const bool none = !(sum != 0.0f);  // NaN is a sum
    if (splits == 1) {
        const float inv = none ? 0.0f : 1.0f / sum, l2 = none ? -INFINITY : ref - kBias + log2_fast(sum);
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int w = 16 * r + 4 * g + i;
                if (w < D / 8) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = run.o[r][j][i] * inv;
                    kv_store8(type, a.out, q.at_row(a.ld_out) + 8 * w, v);
                }
            }
        if (g == 0) attend_lse(a, sp.lse2, q.out_row(a), l2);
    } else {
        const int64_t row = (((int64_t)split * tiles.live + place) * a.c.heads + head) * sp.few_rows + n;
        if (g == 0) sp.few_stats[row] = make_float2(ref == -INFINITY ? ref : ref - kBias, sum);
        if (none) return;
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int w = 16 * r + 4 * g + i;
                if (w < D / 8) {
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = run.o[r][j][i];
                    kv_store8<0>(sp.few_sums, row * D + 8 * w, v);
                }
            }
    }
}

// The splits of a row joined.  Rows of k_attend have LANES threads (64, or 256 for rows of
// many splits): thread t of them has elements 8 (t % (D/8)) .. of the splits t / (D/8), +
// groups, ..; the groups' sums are added in their order.  The workgroups from few_blocks on
// have rows of k_attend_rows, which are many and of few splits: a thread has four elements
// of a row and adds up all splits (14000 rows of 64 elements in 4 splits: 17.2 us with a
// wavefront a row, 9.5 that way).
template <int ROWS>
__device__ __forceinline__ int join_row(const AttendArgs &a, const Splits &sp, int first, int at, int64_t &out_row, int64_t &rows) {
    constexpr bool many = ROWS == kManyTile;
    Tiles<ROWS> tiles;
    tiles.open(a, sp);
    const int per = many ? ROWS : sp.few_rows, x = first / per, place = x / a.c.heads, head = x - place * a.c.heads;
    rows = (int64_t)tiles.live * a.c.heads * per;
    int b, tile;
    KvRows k;
    if (tiles.splits == 1 || place >= tiles.live || !tiles.place(a, place, b, tile, k)) return 0;
    const int row = tile * ROWS + at - x * per;
    if (row >= k.count * a.group) return 0;
    out_row = attend_out_row(a, k, head, row);
    return tiles.splits;
}
__device__ __forceinline__ void join_many(const AttendArgs &a, const Splits &sp, int type, int block) {
    const int D = a.c.D, lanes = D <= 64 ? 16 : (D <= 128 ? 32 : 64);  // a row's
    const int first = block * (kThreads / lanes), row = first + threadIdx.x / lanes, e = threadIdx.x % lanes;  // of one tile
    int64_t out_row, rows;
    const int n = join_row<kManyTile>(a, sp, first, row, out_row, rows);
    if (n == 0 || 4 * e >= D) return;
    float ref = -INFINITY, sum = 0.0f;
    f4 v = {0, 0, 0, 0};
#pragma unroll 4
    for (int s = 0; s < n; ++s) ref = fmaxf(ref, sp.many_stats[s * rows + row].x);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
        const float2 st = sp.many_stats[s * rows + row];
        const f4 u = *reinterpret_cast<const f4 *>(sp.many_sums + (s * rows + row) * D + 4 * e);
        // a sum of 0: nothing was seen, and nothing written
        const float f = st.y == 0.0f ? 0.0f : (st.x == -INFINITY ? 1.0f : exp2_fast(st.x - ref));
        if (f != 0.0f) {
            sum = fmaf(st.y, f, sum);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fmaf(u[j], f, v[j]);
        }
    }
    const bool none = !(sum != 0.0f);
    const float inv = none ? 0.0f : 1.0f / sum;
    attend_store4(type, a.out, attend_at(a, out_row, a.ld_out) + 4 * e, v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    if (e == 0) attend_lse(a, sp.lse2, out_row, none ? -INFINITY : ref + log2_fast(sum));
}
template <int LANES>
__global__ __launch_bounds__(kThreads) void k_attend_join(AttendArgs a, Splits sp, int type, int few_rows, int few_blocks) {
    if ((int)blockIdx.x >= few_blocks) {
        join_many(a, sp, type, blockIdx.x - few_blocks);
        return;
    }
    __shared__ float part[kThreads * 8];
    __shared__ float weight[kThreads], by[kThreads];
    const int D = a.c.D, each = D / 8, groups = LANES / each;
    const int tid = threadIdx.x % LANES, base = threadIdx.x - tid;
    const int row = blockIdx.x * (kThreads / LANES) + __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
    const float *sums = sp.few_sums;
    const float2 *stats = sp.few_stats;
    int64_t out_row, rows;
    const int n = row < few_rows ? join_row<kFewTile>(a, sp, row, row, out_row, rows) : 0;
    // a row's threads are one wavefront or the workgroup
    auto sync = [] {
        if (LANES > 64) __syncthreads();
        else {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    };
    if (n == 0) return;
    // n <= LANES splits: a thread has one's reference and sum
    float2 st = make_float2(-INFINITY, 0.0f);
    if (tid < n) st = stats[tid * rows + row];
    const int s0 = tid / each, e = tid - s0 * each;
    constexpr int FIRST = 4;  // of the thread's splits, on their way meanwhile (what was not written is not used)
    float first[FIRST][8];
#pragma unroll
    for (int i = 0; i < FIRST; ++i)
        if (s0 < groups && s0 + i * groups < n) kv_load8<0>(sums, ((s0 + i * groups) * rows + row) * D + 8 * e, first[i]);
    float ref = st.x, sum = 0.0f, v[8] = {};
    for (int o = 1; o < 64; o <<= 1) ref = fmaxf(ref, __shfl_xor(ref, o, 64));
    if (LANES > 64) {
        if ((tid & 63) == 0) weight[threadIdx.x] = ref;
        sync();
        for (int w = 0; w < LANES / 64; ++w) ref = fmaxf(ref, weight[base + 64 * w]);
        sync();
    }
    const bool some = st.y != 0.0f;  // else nothing was seen, and nothing written
    by[threadIdx.x] = !some ? 0.0f : (st.x == -INFINITY ? 1.0f : exp2_fast(st.x - ref));
    weight[threadIdx.x] = some ? st.y * by[threadIdx.x] : 0.0f;
    sync();
    auto add = [&](int s, const float (&u)[8]) {
        const float f = by[base + s];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = f != 0.0f ? fmaf(u[j], f, v[j]) : v[j];
    };
    if (s0 < groups) {
#pragma unroll
        for (int i = 0; i < FIRST; ++i)
            if (s0 + i * groups < n) add(s0 + i * groups, first[i]);
#pragma unroll 4
        for (int s = s0 + FIRST * groups; s < n; s += groups) {
            float u[8];
            kv_load8<0>(sums, (s * rows + row) * D + 8 * e, u);
            add(s, u);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j * kThreads + threadIdx.x] = v[j];
    sync();
    if (tid >= each) return;
    for (int s = 1; s < groups && s < n; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += part[j * kThreads + base + s * each + tid];
    for (int s = 0; s < n; ++s) sum += weight[base + s];
    const bool none = !(sum != 0.0f);
    const float inv = none ? 0.0f : 1.0f / sum, l2 = none ? -INFINITY : ref + log2_fast(sum);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= inv;
    kv_store8(type, a.out, attend_at(a, out_row, a.ld_out) + 8 * tid, v);
    if (tid == 0) attend_lse(a, sp.lse2, out_row, l2);
}

// The weight that each entry got, for sequences of few rows: mass[j] += sum over rows and
// heads of the group of 2^(x - lse2).  A wavefront owns 32 entries of a head and goes
// over the rows, 16 at a time, so every place is added to by one lane, in a fixed order.
// A chain of latencies (table, codes, queries, lse) that little overlaps, and the keys are read and decoded a second
// time: 16 sequences of 4000 entries, 8 heads of 128, one token of 4 query heads each add 37 us to 30, their bytes 8.
template <int PIECES, int D>
__global__ __launch_bounds__(kThreads) void k_attend_mass(AttendArgs a, Splits sp, int type, int tiles) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
    const int head = blockIdx.x % a.c.heads, x = blockIdx.x / a.c.heads, b = x / tiles;
    const int k0 = ((x - b * tiles) * kWaves + wave) * kKeys;
    const KvRows rows = kv_rows(a.c, b);
    if (k0 >= rows.len || rows.count == 0 || rows.count * a.group > kMassRoom) return;
    Step<D> t;
    read_step<D>(a.c, b, head, k0, (rows.len - 1) & ~15, t);
    Decode decode;
    decode.set();
    // rows that see any of these entries
    const int shift = rows.len - rows.count;
    int i0 = a.causal ? k0 - shift : 0, i1 = a.window > 0 ? k0 + kKeys - 1 + a.window - shift : rows.count;
    i0 = i0 < 0 ? 0 : i0;
    i1 = i1 > rows.count ? rows.count : i1;
    float got[8] = {};
    for (int tile = i0 * a.group / kRows; tile * kRows < i1 * a.group; ++tile) {
        Tile<PIECES, D> q;
        q.type = type;
        if (!q.open(a, b, rows, tile, head)) break;
        q.queries(a);
        float p[8];
        products<PIECES, D>(decode, t, q.q, p);
        const float lse = sp.lse2[attend_group_row(a, q.batch_row, head, q.q_head - head * a.group)];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = k0 + 16 * (i >> 2) + 4 * g + (i & 3);
            if (q.live && lse != -INFINITY && at >= q.lo && at < q.hi) got[i] += exp2_fast(fmaf(p[i], q.factor, -lse));
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) got[i] += __shfl_xor(got[i], o, 64);
        const int at = k0 + 16 * (i >> 2) + 4 * g + (i & 3);
        if (n == 0 && at < rows.len) a.mass[((int64_t)b * a.c.heads + head) * a.ld_mass + at] += got[i];
    }
}

// ---- the shape of a call, from what the host knows
struct Shape {
    Splits sp;
    int64_t few_groups, many_groups;  // workgroups; many_groups 0: no sequence has so many rows
    int64_t few_parts, many_parts;    // rows that have parts, times splits
    int64_t few_join, many_join;      // rows that are joined
    bool mass_rows;                   // whether a sequence can have more than kMassRoom
    int64_t bytes;                    // of the workspace
};
constexpr int64_t quads(int64_t floats) { return (floats + 3) / 4 * 4; }  // whole 16 bytes of a workspace

// The most rows of a sequence and head that k_attend takes.  It decodes the entries anew for every 16 rows, and
// k_attend_rows for every 256, which pays once enough of these have rows.  us with up to 32 rows here and with all (8 cache
// heads, 4 query heads of each, out alone):
//                             256 rows    512 rows    768 rows    1024 rows    2048 rows    8192 rows
//   bf16, D =  64, 2 x 4096    44   39     50   59     57   73     62    88     94   149    226   427
//         D = 128, 2 x 4096    57   44     61   69     71   85     80   102    120   175    283   511
//                 16 x 4000   121  179    184  332    335  475    348   624    652  1175   2076  3714
//         D = 192, 2 x 4096    77   60     88   95    107  134    121   167    195   304    464   935
//                 16 x 4000   197  307    301  595    562  866    572  1141   1156  2200   3597  7093
//   fp32, D =  64, 2 x 4096    56   49     61   76     74   96     84   115    134   195    347   575
//         D = 128, 2 x 4096    76   51     83   78    106  100    126   127    210   223    562   676
//                  4 x 4000    82   76    125  127    186  175    208   224    355   413   1068  1308
//                 16 x 4000   208  228    361  432    638  626    699   829   1343  1593   4181  5048
// Which is better turns on the tiles that fill the GPU too; rows alone are what the host knows.
constexpr int64_t kAnyRows = 0x7fffffff;
int64_t few_room(int type, int64_t D) { return attend_rows_has(type, D) ? (type == 0 ? 768 : 256) : kAnyRows; }

// largest: no call's shape but one whose workspace is no smaller than that of any call of up to T rows and B sequences,
// with starts or without: for as many sequences as are split, however many tiles are sure to have rows.
Shape shape_of(int type, int64_t T, int64_t B, int64_t capacity, int64_t heads, int64_t group, int64_t D, bool ragged, bool mass,
               bool largest = false) {
    Shape p{};
    if (largest && ragged && B > kCounted) B = kCounted;
    const int64_t rows = T * group, room = ragged ? few_room(type, D) : kAnyRows;
    const int64_t few = largest ? kAnyRows : room;  // rows of a sequence that k_attend can have: without starts any
    p.sp.few_room = (int)room;
    p.sp.few_rows = (int)(!ragged && group < kFewTile ? group : kFewTile);
    auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
    // Tiles that can have rows.  As many workgroups as the GPU holds at once, but no split below one step of each of
    // their wavefronts, and splits that a joining wavefront has a lane for, unless there are few rows.  sure: tiles
    // that have rows for certain.
    auto share = [&](int64_t tiles, int64_t sure, int64_t at_once, int64_t step, int per, int &most_tiles, int &want, int &most,
                     int64_t &groups, int64_t &parts, int64_t &join) {
        const int64_t fit = at_once / heads > 1 ? at_once / heads : 1, steps = (capacity + step - 1) / step;
        most_tiles = (int)tiles;
        want = (int)fit;
        most = (int)least(least(steps, fit), tiles * heads <= at_once / 64 ? 256 : 64);
        if (!largest && ((ragged && B > kCounted) || fit < 2 * sure)) most = 1;
        groups = least(fit > tiles ? fit : tiles, tiles * most) * heads;
        parts = most > 1 ? least(fit, tiles * most) * heads * per : 0;
        join = most > 1 ? least(tiles, fit / 2) * heads * per : 0;
    };
    const int64_t each = D > 128 ? at_once<1, 256> : (type == 0 && D == 128 ? at_once<2, 128> : at_once<1, 128>);
    const int64_t apart = B * ((least(few, rows) + kFewTile - 1) / kFewTile), packed = rows / kFewTile + B;
    share(!ragged ? B * ((group + kFewTile - 1) / kFewTile) : (B > kCounted ? packed : least(apart, packed)), 0, 256 * each,
          kKeys * kWaves, p.sp.few_rows, p.sp.few_tiles, p.sp.few_want, p.sp.few_most, p.few_groups, p.few_parts, p.few_join);
    if (ragged && rows > room)
        share(rows / kManyTile + (B > kCounted ? B : least(B, rows / room)), rows > B * room ? (rows - B * room) / kManyTile : 0,
              256, 512, kManyTile, p.sp.many_tiles, p.sp.many_want, p.sp.many_most, p.many_groups, p.many_parts, p.many_join);
    const int64_t parts = p.few_parts + p.many_parts, all = quads(rows * heads);
    p.bytes = parts * D * 4 + quads(parts * 2) * 4 + (mass ? all * 4 : 0);
    p.mass_rows = mass && (ragged ? rows : group) > kMassRoom;
    if (p.mass_rows) {
        p.sp.query_piece = all * D;
        p.bytes += all * D * 2 * (type == 0 ? 2 : 1) + all * 4;
    }
    return p;
}
Shape shape_of(int type, const AttendArgs &a) {
    Shape p = shape_of(type, a.c.T, a.c.B, (int64_t)a.c.width << a.c.page_log2, a.c.heads, a.group, a.c.D, a.c.starts != nullptr,
                       a.mass != nullptr);
    float *at = a.ws;
    p.sp.few_sums = at;
    at += p.few_parts * a.c.D;
    p.sp.many_sums = at;
    at += p.many_parts * a.c.D;
    p.sp.few_stats = reinterpret_cast<float2 *>(at);
    p.sp.many_stats = p.sp.few_stats + p.few_parts;
    if (a.mass == nullptr) return p;
    at += quads((p.few_parts + p.many_parts) * 2);
    const int64_t all = quads((int64_t)a.c.T * a.c.heads * a.group);
    p.sp.lse2 = at;
    at += all;
    if (p.mass_rows) {
        p.sp.factors = at;
        p.sp.queries = reinterpret_cast<_Float16 *>(at + all);
    }
    return p;
}
// workgroups of k_attend_mass per sequence and head; attend_mass.hip's take half as many entries
int64_t mass_tiles(const AttendArgs &a) {
    return (((int64_t)a.c.width << a.c.page_log2) + kKeys * kWaves - 1) / (kKeys * kWaves);
}

template <int PIECES, int WP, int D>
hipError_t launch(int type, const AttendArgs &a, const Shape &p, hipStream_t s) {
    constexpr int bytes = kWaves * Ring<D>::WAVE;
    static std::atomic<uint64_t> lds_set{0};
    hipError_t e = ensure_lds_bytes((const void *)k_attend<PIECES, WP, D>, bytes, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attend<PIECES, WP, D>), dim3((unsigned)p.few_groups), dim3(kThreads), bytes, s, a, p.sp, type);
    e = hipGetLastError();
    if (e == hipSuccess && p.many_groups) e = launch_attend_rows(type, a, p.sp, p.many_groups, s);
    if (e == hipSuccess && p.few_join + p.many_join) {
        const int64_t lanes = D <= 64 ? 16 : (D <= 128 ? 32 : 64), many = p.many_join / (kThreads / lanes);
        // few rows of many splits: a workgroup each
        if (p.sp.few_most > 64 || p.few_join <= 512)
            hipLaunchKernelGGL(k_attend_join<kThreads>, dim3((unsigned)(p.few_join + many)), dim3(kThreads), 0, s, a, p.sp, type,
                               (int)p.few_join, (int)p.few_join);
        else
            hipLaunchKernelGGL(k_attend_join<64>, dim3((unsigned)((p.few_join + 3) / 4 + many)), dim3(kThreads), 0, s, a, p.sp,
                               type, (int)p.few_join, (int)((p.few_join + 3) / 4));
        e = hipGetLastError();
    }
    if (e != hipSuccess || a.mass == nullptr) return e;
    if (p.mass_rows) e = launch_attend_mass_rows(type, a, p.sp, s);
    if (e != hipSuccess) return e;
    const int64_t per = mass_tiles(a);
    hipLaunchKernelGGL((k_attend_mass<PIECES, D>), dim3((unsigned)(a.c.B * per * a.c.heads)), dim3(kThreads), 0, s, a, p.sp,
                       type, (int)per);
    return hipGetLastError();
}

template <int PIECES, int WP>
hipError_t launch_for(int type, const AttendArgs &a, const Shape &p, hipStream_t s) {
    switch (a.c.D) {
        case 64: return launch<PIECES, WP, 64>(type, a, p, s);
        case 96: return launch<PIECES, WP, 96>(type, a, p, s);
        case 128: return launch<PIECES, WP, 128>(type, a, p, s);
        case 192: return launch<PIECES, WP, 192>(type, a, p, s);
        default: return launch<PIECES, WP, 256>(type, a, p, s);
    }
}

}  // namespace

int64_t attend_workspace_bytes(int type, int64_t T, int64_t B, int64_t capacity, int64_t heads, int64_t group, int64_t D,
                               bool ragged, bool mass) {
    return shape_of(type, T, B, capacity, heads, group, D, ragged, mass, true).bytes;
}

int64_t attend_workspace_used(int type, const AttendArgs &a) { return shape_of(type, a).bytes; }

void attend_shape(int type, const AttendArgs &a, int *few, int *many) {
    const Shape p = shape_of(type, a);
    *few = p.sp.few_most;
    *many = p.many_groups ? p.sp.many_most : 0;
}

bool attend_grid_ok(int type, const AttendArgs &a) {
    constexpr int64_t most = (int64_t(1) << 24) - 1;  // workgroups of 256 threads; half as many of 512
    const Shape p = shape_of(type, a);
    return p.few_groups <= most && p.many_groups <= most / 2 && p.few_join + p.many_join <= most &&
           (a.mass == nullptr || a.c.B * mass_tiles(a) * a.c.heads <= most / 2);
}

hipError_t launch_attend(int type, const AttendArgs &a, hipStream_t s) {
    const Shape p = shape_of(type, a);
    if (type == 0) return launch_for<2, 2>(type, a, p, s);
    return type == 1 ? launch_for<1, 2>(type, a, p, s) : launch_for<1, 1>(type, a, p, s);
}

}  // namespace qmm
