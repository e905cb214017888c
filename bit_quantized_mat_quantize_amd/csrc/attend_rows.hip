// attend_rows.hip -- attention over the paged 4-bit cache, many rows per sequence
// (gfx950): prompts, and parts of them.
//
// A workgroup takes a tile of query rows (row = token * group + head of the group: 32 per
// wavefront) and one cache head, and goes over the entries that any of them sees, KT at a
// time.  The entries are decoded once per workgroup, to fp16 in LDS, keys as [entry][element]
// and values as [element][entry], a tile ahead of the one that is multiplied; its codes
// come from memory while that one is.  Then, per wavefront and 32 entries,
//
//   S^T = K Q^T    (32 entries x 32 rows, on 32x32x16 matrix instructions)
//   O^T += V^T P^T
//
// with the entries along the registers and the rows along the lanes in both, so that P
// needs no exchange between lanes: the order in which a lane's registers hold the
// entries is the order of the values in LDS.
//
// Of 16-bit queries, values and P are rounded to fp16.  Keys, scale * code of up to 14 bits, are
// two fp16 pieces, exact, for fp16 queries and where lse or mass are asked for: rounded to one
// they put fp16 outputs at 4.4e-4 of the norm from the 64-bit result where fp16 itself costs
// 2.1e-4 (now 2.9e-4; 9 sequences, 555 rows, window 1024), moved weights by per cents with scores of
// hundreds, and would show in lse and mass.  For bf16 outputs alone they are rounded: these are 1.7e-3 off either
// way, and two pieces are half as many matrix instructions again (2 prompts of 2048 rows on
// 8192 entries each, 32 heads of 128: 695 us and 847).  fp32 queries, and with them the
// decoded entries and P, are two fp16 pieces each (22 bits), of whose four products the three
// large ones are taken.  All scales of a workgroup are multiplied by one power of two for the
// keys and one for the values, which move when a larger scale turns up (then the tile is
// decoded again; after the first tile that is seldom).
//
// Bounds: matrix and vector instructions, which overlap in part only (of the cycles, 2 prompts
// of 2048 rows on 8192 entries, 32 heads of 128 in bf16: 32% and 42%; 525 to 549 us a call
// from card to card, 800 TFLOP/s; fp32, 3 of 700 rows on 2100 entries, 28 heads: 29% and
// 22%, 200 us, waiting for one another's steps).  256 rows are what the registers of
// two wavefronts a SIMD hold; of half as many rows the decode would weigh twice as much.
// The two halves of a workgroup taking turns, one multiplying while the other forms
// weights, took 730 us.
#include "attend_device.h"

namespace qmm {
namespace {

// Rows of a tile, entries of a step.
// KP: pieces of a key.  PIECES: of a query, a weight and a value.
template <int KP, int PIECES, int D>
struct Shape {
    static constexpr int WAVES = 8, KT = 64, ROWS = kManyTile, THREADS = 64 * WAVES;
    static_assert(ROWS == 32 * WAVES, "32 rows a wavefront");
    static constexpr int NB = D / 32, WORDS = D / 8, ROUNDS = D > 128 ? 2 : 1;
    static constexpr int KEY_ROW = D == 96 ? 128 : D;              // elements of a key's row in LDS
    static constexpr int KEYS = KT * KEY_ROW * 2, VALUES = D * KT * 2;  // bytes of one piece
    static constexpr int STAGE = KP * KEYS + PIECES * VALUES, BYTES = 2 * STAGE;
    static constexpr int GROUPS = 2 * KT / 16, MINE = GROUPS / WAVES;  // groups of 16 entries' keys or values; per wavefront
    static_assert(MINE == 1, "one group per wavefront");
    // a group on its way: 16 * D/2 bytes of codes, D/32 * 32 of scales
    static constexpr int CODE_LOADS = (8 * D + 1023) / 1024, LOADS = CODE_LOADS + 1;
    static constexpr int RAW = 9 * D;
    static constexpr int ROOM = 160 * 1024 - 512 - BYTES;  // of LDS
    static constexpr int SLOTS = ROOM >= 3 * WAVES * RAW ? 3 : (ROOM >= 2 * WAVES * RAW ? 2 : 1);
    static constexpr int ALL = BYTES + SLOTS * WAVES * RAW;
    static_assert(ALL + 512 <= 160 * 1024, "LDS");
};

// 16-byte pieces of LDS rows are placed so that eight lanes of one access meet eight of them
template <int D>
__device__ __forceinline__ int key_piece(int entry, int w) {
    return entry * Shape<1, 1, D>::KEY_ROW * 2 + ((w ^ (entry & 7)) * 16);
}
template <int D>
__device__ __forceinline__ int value_piece(int element, int c) {  // c: eight entries
    constexpr int KT = Shape<1, 1, D>::KT;
    const int by = (element ^ (element >> 3)) & 7;
    return element * KT * 2 + ((c ^ by) * 16);
}

// what a lane decodes of its group
template <int D>
struct Raw {
    static constexpr int NB = D / 32, ROUNDS = D > 128 ? 2 : 1;
    uint32_t w[ROUNDS * 4];              // keys: the words of all blocks; values: a word of four entries
    uint32_t s[NB > 2 * ROUNDS ? NB : 2 * ROUNDS];  // keys: scales of all blocks; values: of four entries
};

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

template <int KP, int PIECES, int D>
__global__ __launch_bounds__((Shape<KP, PIECES, D>::THREADS), 1) void k_attend_rows(AttendArgs a, Splits sp, int type) {
    using S = Shape<KP, PIECES, D>;
    constexpr int NB = S::NB, KT = S::KT, WORDS = S::WORDS, ROUNDS = S::ROUNDS;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ uint32_t flags[10];
    uint32_t(*largest)[2] = reinterpret_cast<uint32_t(*)[2]>(flags);    // [stage][keys, values]: the bits of scales beyond the bound
    uint32_t(*unfit)[2] = reinterpret_cast<uint32_t(*)[2]>(flags + 4);  // [step % 3]: entries that make NaN, a bit each
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, hf = lane >> 5;
    const int head = blockIdx.x % a.c.heads, x = blockIdx.x / a.c.heads;
    Tiles<S::ROWS> tiles;
    tiles.open(a, sp);
    const int splits = tiles.splits, place = tiles.live - 1 - x / splits, split = x % splits;  // later rows see more: first
    int b, tile;
    KvRows rows;
    if (place < 0 || !tiles.place(a, place, b, tile, rows)) return;
    const int total = rows.count * a.group;
    if (total <= sp.few_room || tile * S::ROWS >= total) return;
    const int r0 = tile * S::ROWS, r1 = r0 + S::ROWS - 1 < total ? r0 + S::ROWS - 1 : total - 1;

    // ---- this lane's row
    const int wr0 = r0 + 32 * wave, wr1 = wr0 + 31 < total ? wr0 + 31 : total - 1;  // the wavefront's
    const bool busy = wr0 < total, live = wr0 + n < total;
    const int use = live ? wr0 + n : r1;
    int lo, hi, first, last, seen0, seen1, all0, all1, unused;
    attend_span(a, rows, use / a.group, lo, hi);
    attend_span(a, rows, r0 / a.group, first, unused);   // entries that the tile sees: [first, last)
    attend_span(a, rows, r1 / a.group, unused, last);
    attend_span(a, rows, (busy ? wr0 : r1) / a.group, seen0, all1);  // that the wavefront sees: [seen0, seen1)
    attend_span(a, rows, (busy ? wr1 : r1) / a.group, all0, seen1);  // that all its rows see: [all0, all1)
    const int token = use / a.group, q_head = head * a.group + use - token * a.group;
    const int64_t out_row = (int64_t)(rows.first + token) * (a.c.heads * a.group) + q_head;
    const int64_t q_at = (int64_t)(rows.first + token) * a.ld_q + (int64_t)q_head * D;
    // ---- this split's steps
    const int s0 = (first < 0 ? 0 : first) / KT, s1 = last > 0 ? (last + KT - 1) / KT : 0, all = s1 > s0 ? s1 - s0 : 0;
    const int from = s0 + (int)((int64_t)all * split / splits), to = s0 + (int)((int64_t)all * (split + 1) / splits);
    const int last16 = last > 0 ? (last - 1) & ~15 : 0;

    // ---- staging.  Group g < KT / 16: keys of its 16 entries, else values.  Lane of a key group: entry
    // lane / 4, word lane % 4 of every block.  Lane of a value group: word w (and w + 16) of
    // entries 4 e .. 4 e + 3.
    const bool keys = wave < KT / 16;
    const int group = keys ? wave : wave - KT / 16;
    const int ke = lane >> 2, kg = lane & 3;
    const int vw = (lane & 7) | ((lane >> 4) & 1) << 3, ve = ((lane >> 3) & 1) << 1 | lane >> 5;
    Decode decode;
    decode.set();
    typedef const __attribute__((address_space(4))) int32_t *scalar_ints;
    const scalar_ints table = (scalar_ints)(uintptr_t)(a.c.table + (int64_t)b * a.c.width);
    // Direct loads into this wavefront's slots, SLOTS steps ahead: the codes of a group are one run of
    // memory, and a lane's place in it is fixed.
    constexpr int SLOTS = S::SLOTS;
    uint8_t *const ring = lds + S::BYTES + wave * (SLOTS * S::RAW);
    const uint32_t ring_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ring);
    uint32_t code_at[S::CODE_LOADS];
#pragma unroll
    for (int i = 0; i < S::CODE_LOADS; ++i) code_at[i] = 16 * (64 * i + lane);
    const uint32_t scale_at = ((D / 2) << a.c.page_log2) + 2 * ((lane >> 3) << a.c.page_log2) + 4 * (lane & 7);  // 4 bytes
    const uint32_t records = (uint32_t)kv_chunk_bytes(a.c);
    uint32_t missing = 0;  // steps whose page is not in the pool, the next one lowest
    auto load = [&](int step, int ahead) {  // ahead: of the step that is multiplied
        int at = step * KT + 16 * group;
        at = at < last16 ? at : last16;
        int page = table[at >> a.c.page_log2];
        const bool none = page < 0 || page >= a.c.pages;
        if (none) page = 0;
        missing |= (none ? 1u : 0u) << ahead;
        const uint64_t base = (uint64_t)(uintptr_t)kv_chunk(a.c, page, keys ? 0 : 1, head);
        const u32x4 r = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, records, 0x00020000u};
        const int e0 = at & ((1 << a.c.page_log2) - 1);
        const uint32_t to = ring_at + ((step - from) % SLOTS) * S::RAW;
#pragma unroll
        for (int i = 0; i < S::CODE_LOADS; ++i)  // lanes behind the group's end are off: they would write to LDS too
            if (64 * i + 64 <= D / 2 || lane < D / 2 - 64 * i)
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(to + 1024 * i),
                             "v"(code_at[i]), "s"(r), "s"(e0 * (D / 2)) : "m0", "memory");
        if (lane < D / 4)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(to + 8 * D),
                         "v"(scale_at), "s"(r), "s"(e0 * 2) : "m0", "memory");
    };
    // the step's group out of its slot, once at most `later` steps' loads behind it are on their way
    auto take = [&](int step, int later, Raw<D> &raw) {
        if (SLOTS > 2 && later >= 2) wait_loads<2 * S::LOADS>();
        else if (SLOTS > 1 && later >= 1) wait_loads<S::LOADS>();
        else wait_loads<0>();
        const uint8_t *slot = ring + ((step - from) % SLOTS) * S::RAW, *scales = slot + 8 * D;
        if (keys) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(slot) + ke * WORDS + kg * NB;
            if constexpr (NB % 4 == 0) {
#pragma unroll
                for (int i = 0; i < NB / 4; ++i) {
                    const uint4 u = ld16(p + 4 * i);
                    raw.w[4 * i] = u.x, raw.w[4 * i + 1] = u.y, raw.w[4 * i + 2] = u.z, raw.w[4 * i + 3] = u.w;
                }
            } else {
#pragma unroll
                for (int i = 0; i < NB; ++i) raw.w[i] = p[i];
            }
#pragma unroll
            for (int i = 0; i < NB; ++i) raw.s[i] = reinterpret_cast<const uint16_t *>(scales)[16 * i + ke];
        } else {
#pragma unroll
            for (int r = 0; r < ROUNDS; ++r) {
                const int w = (16 * r + vw) % WORDS;
                const uint4 u = ld16(slot + (ve * WORDS + w) * 16);
                raw.w[4 * r] = u.x, raw.w[4 * r + 1] = u.y, raw.w[4 * r + 2] = u.z, raw.w[4 * r + 3] = u.w;
                const uint2 d = *reinterpret_cast<const uint2 *>(scales + 32 * (w >> 2) + 8 * ve);
                raw.s[2 * r] = d.x, raw.s[2 * r + 1] = d.y;
            }
        }
    };
    int key_shift = 15, value_shift_ = 15;
    uint32_t key_bound = 0, value_bound = 0;
    auto put = [&](int step, Raw<D> &raw, bool nowhere) {
        uint8_t *stage = lds + (step & 1) * S::STAGE;
        const int e = 16 * group, k0 = step * KT + e;  // in LDS; in the sequence
        constexpr int SCALES = NB > 2 * ROUNDS ? NB : 2 * ROUNDS;
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < SCALES; ++i)
            if (i < (keys ? NB : 2 * ROUNDS)) top = max_u16x2(top, raw.s[i] & 0x7fff7fffu);
        top = (top & 0xffffu) > (top >> 16) ? top & 0xffffu : top >> 16;
        if (k0 < first || k0 + 16 > last || nowhere || __any(top >= (keys ? key_bound : value_bound))) {
            // entries that no row sees are zero, values that are not finite too (their entries' scores are
            // made NaN), and a scale beyond all so far is told to the workgroup
            uint32_t bad = 0;  // bits of the group's 16 entries
            auto keep = [&](uint32_t &s, int i, int at) {  // 16-bit scale i of s, of entry `at` of the group
                const uint32_t m = (s >> (16 * i)) & 0x7fffu;
                const bool out = k0 + at < first || k0 + at >= last;
                if (out || (m >= 0x7c00u && !keys)) s &= i ? 0xffffu : 0xffff0000u;
                if (!out && (nowhere || (m >= 0x7c00u && !keys))) bad |= 1u << at;
                return out || m >= 0x7c00u ? 0u : m;
            };
            top = 0;
#pragma unroll
            for (int i = 0; i < SCALES; ++i)
                if (i < (keys ? NB : 2 * ROUNDS)) {
                    const uint32_t m0 = keys ? keep(raw.s[i], 0, ke) : keep(raw.s[i], 0, 4 * ve + 2 * (i & 1));
                    const uint32_t m1 = keys ? 0u : keep(raw.s[i], 1, 4 * ve + 2 * (i & 1) + 1);
                    top = m0 > top ? m0 : top;
                    top = m1 > top ? m1 : top;
                }
            if (top >= (keys ? key_bound : value_bound)) atomicMax(&largest[step & 1][keys ? 0 : 1], top);
            if (bad) atomicOr(&unfit[step % 3][e >> 5], bad << (e & 31));
        }
        if (keys) {
            const _Float16 unit = (_Float16)pow2i(key_shift);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                const uint32_t ss = raw.s[i] | raw.s[i] << 16;
                const h2 d = as_h2(ss) * h2{unit, unit};
                const uint32_t w = raw.w[i];
                const h2 c[4] = {centred_even(decode.even(w)), centred_odd(decode.odd(w)), centred_even(decode.even(w >> 8)),
                                 centred_odd(decode.odd(w >> 8))};
                h2 h[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = c[j] * d;
                uint8_t *to = stage + key_piece<D>(e + ke, 4 * i + kg);
                *reinterpret_cast<uint4 *>(to) = make_uint4(as_u32(h[0]), as_u32(h[1]), as_u32(h[2]), as_u32(h[3]));
                if constexpr (KP == 2) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) h[j] = __builtin_elementwise_fma(c[j], d, -h[j]);
                    *reinterpret_cast<uint4 *>(to + S::KEYS) =
                        make_uint4(as_u32(h[0]), as_u32(h[1]), as_u32(h[2]), as_u32(h[3]));
                }
            }
        } else {
            stage += KP * S::KEYS;
            const _Float16 unit = (_Float16)pow2i(value_shift_);
#pragma unroll
            for (int r = 0; r < ROUNDS; ++r) {
                const int w = 16 * r + vw;
                const h2 d[2] = {as_h2(raw.s[2 * r]) * h2{unit, unit}, as_h2(raw.s[2 * r + 1]) * h2{unit, unit}};
                if (w < WORDS) {
                    // entries 4 ve .. within the eight that a lane of the product holds: 0 and 2, or 1 and 3
                    const int c = 2 * group + (ve & 1), half = (ve >> 1) * 8;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t both[2] = {__builtin_amdgcn_perm(raw.w[4 * r + 1], raw.w[4 * r], 0x0c040c00u + 0x00010001u * y),
                                                  __builtin_amdgcn_perm(raw.w[4 * r + 3], raw.w[4 * r + 2], 0x0c040c00u + 0x00010001u * y)};
#pragma unroll
                        for (int o = 0; o < 2; ++o) {
                            const h2 c0 = o ? centred_odd(decode.odd(both[0])) : centred_even(decode.even(both[0]));
                            const h2 c1 = o ? centred_odd(decode.odd(both[1])) : centred_even(decode.even(both[1]));
                            const h2 h0 = c0 * d[0], h1 = c1 * d[1];
                            uint8_t *to = stage + value_piece<D>(8 * w + 2 * y + o, c) + half;
                            *reinterpret_cast<uint2 *>(to) = make_uint2(as_u32(h0), as_u32(h1));
                            if constexpr (PIECES == 2)
                                *reinterpret_cast<uint2 *>(to + S::VALUES) =
                                    make_uint2(as_u32(__builtin_elementwise_fma(c0, d[0], -h0)),
                                               as_u32(__builtin_elementwise_fma(c1, d[1], -h1)));
                        }
                    }
                }
            }
        }
    };

    // ---- the rows' running results
    f16v o[NB];   // o[block][4 i + r]: element 32 block + 8 i + 4 hf + r of row n, times 2^value_shift (16-fold for odd r)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    float ref = -INFINITY, sum = 0.0f;
    auto scale = [&](float by) {
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] *= by;
    };

    if (threadIdx.x < 10) flags[threadIdx.x] = 0;
    __syncthreads();
    // The two wavefronts of a SIMD would all multiply, or all form weights, at the same time; with
    // one ahead of the other, its weights are formed while the other multiplies.
    if (wave < S::WAVES / 2) __builtin_amdgcn_s_setprio(1);
    Raw<D> raw;
    for (int i = 0; i < SLOTS; ++i)
        if (from + i < to) load(from + i, i);
    // ---- the rows' queries, while the first entries are on their way
    h8 qh[2 * NB], ql[PIECES == 2 ? 2 * NB : 1];  // elements 16 i + 8 hf ..
    float factor;
    {
        const int64_t at = q_at + 8 * hf;
        uint32_t top = 0;
        float f[8];
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
            kv_load8(type, a.q, at + 16 * i, f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t u = __float_as_uint(f[j]) & 0x7fffffffu;
                top = u > top ? u : top;
            }
        }
        const uint32_t other = __shfl_xor(top, 32, 64);
        top = other > top ? other : top;
        const int shift = query_shift(top);
        const float by = a.scale < 0.0f ? -pow2i(shift) : pow2i(shift);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {
            kv_load8(type, a.q, at + 16 * i, f);
            query_pieces<PIECES>(f, by, qh[i], ql[PIECES == 2 ? i : 0]);
        }
        factor = (top >> 23) == 255 ? __builtin_nanf("") : fabsf(a.scale) * pow2i(-shift);
        if (sp.queries != nullptr && split == 0 && live) {  // for the weights of the entries
            const int64_t row = attend_group_row(a, rows.first, head, use);
#pragma unroll
            for (int i = 0; i < 2 * NB; ++i) {
                _Float16 *p = sp.queries + row * D + 16 * i + 8 * hf;
                *reinterpret_cast<h8 *>(p) = qh[i];
                if constexpr (PIECES == 2) *reinterpret_cast<h8 *>(p + sp.query_piece) = ql[i];
            }
            if (hf == 0) sp.factors[row] = factor;
        }
    }

    auto behind = [&](int step) { return to - 1 - step < SLOTS - 1 ? to - 1 - step : SLOTS - 1; };
    if (from < to) {
        take(from, behind(from), raw);
        put(from, raw, missing & 1);
    }
    for (int step = from; step < to; ++step) {
        __syncthreads();  // the step's entries are in LDS, and nobody reads the step's before
        const uint8_t *stage = lds + (step & 1) * S::STAGE;
        const uint32_t top[2] = {largest[step & 1][0], largest[step & 1][1]};
        if (top[0] >= key_bound || top[1] >= value_bound) {
            // the same for the whole workgroup: a larger scale than all before
            if (top[0] >= key_bound) {
                key_shift = value_shift(top[0]);
                key_bound = ((top[0] >> 10) + 1) << 10;
            }
            if (top[1] >= value_bound) {
                const int shift = value_shift(top[1]);
                scale(pow2i(shift - value_shift_));
                value_shift_ = shift;
                value_bound = ((top[1] >> 10) + 1) << 10;
            }
            __syncthreads();
            take(step, behind(step), raw);
            put(step, raw, missing & 1);
            __syncthreads();
        }
        if (threadIdx.x < 2) unfit[(step + 2) % 3][threadIdx.x] = 0;
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot's reads are done
        if (step + SLOTS < to) load(step + SLOTS, SLOTS);
        missing >>= 1;
        if (busy) {
            const float by = factor * pow2i(-key_shift);
#pragma unroll
            for (int sub = 0; sub < KT / 32; ++sub) {
                const int k0 = step * KT + 32 * sub;
                if (k0 >= seen1 || k0 + 32 <= seen0) continue;  // the same for the wavefront
                f16v x;
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    const uint8_t *p = stage + key_piece<D>(32 * sub + n, 2 * i + hf);
                    const h8 kh = *reinterpret_cast<const h8 *>(p);
                    x = mfma32(kh, qh[i], x);
                    if constexpr (PIECES == 2) x = mfma32(kh, ql[i], x);
                    if constexpr (KP == 2) {
                        const h8 kl = *reinterpret_cast<const h8 *>(p + S::KEYS);
                        x = mfma32(kl, qh[i], x);
                    }
                }
                const uint32_t bad = __builtin_amdgcn_readfirstlane(unfit[step % 3][sub]);
                if (__builtin_expect(bad != 0, 0)) {
                    asm volatile("");  // not worth a select per score
#pragma unroll
                    for (int r = 0; r < 16; ++r)
                        if ((bad >> (8 * (r >> 2) + 4 * hf + (r & 3))) & 1) x[r] = __builtin_nanf("");
                }
                float f = by;
                if (k0 < all0 || k0 + 32 > all1) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int at = k0 + 8 * (r >> 2) + 4 * hf + (r & 3);
                        x[r] = at < lo || at >= hi ? -INFINITY : x[r] * by;
                    }
                    f = 1.0f;
                }
                float most = x[0];
#pragma unroll
                for (int r = 1; r < 16; ++r) most = fmaxf(most, x[r]);
                most *= f;
                if (__any(most > ref + kSlack)) {
                    most = fmaxf(most, __shfl_xor(most, 32, 64));
                    const float next = fmaxf(ref, most), down = next == -INFINITY ? 1.0f : exp2_fast(ref - next);
                    scale(down);
                    sum *= down;
                    ref = next;
                }
                const float less = ref == -INFINITY ? 0.0f : kBias - ref;
                h8 ph[2], pl[2];
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const float p = exp2_fast(fmaf(x[r], f, less));
                    sum += p;
                    ph[r >> 3][r & 7] = (_Float16)p;
                    if constexpr (PIECES == 2) pl[r >> 3][r & 7] = (_Float16)(p - (float)ph[r >> 3][r & 7]);
                }
#pragma unroll
                for (int i = 0; i < NB; ++i)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint8_t *p = stage + KP * S::KEYS + value_piece<D>(32 * i + n, 2 * (2 * sub + t) + hf);
                        const h8 vh = *reinterpret_cast<const h8 *>(p);
                        o[i] = mfma32(vh, ph[t], o[i]);
                        if constexpr (PIECES == 2) {
                            const h8 vl = *reinterpret_cast<const h8 *>(p + S::VALUES);
                            o[i] = mfma32(vh, pl[t], o[i]);
                            o[i] = mfma32(vl, ph[t], o[i]);
                        }
                    }
            }
        }
        if (step + 1 < to) {
            take(step + 1, behind(step + 1), raw);
            put(step + 1, raw, missing & 1);
        }
    }
    if (!busy) return;
    sum += __shfl_xor(sum, 32, 64);
    if (!live) return;
    const bool none = !(sum != 0.0f);  // NaN is a sum
    const float down = pow2i(-value_shift_);
    if (splits == 1) {
        const float inv = none ? 0.0f : down / sum;
        const int64_t to_row = (int64_t)(rows.first + token) * a.ld_out + (int64_t)q_head * D;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = o[i][4 * c + r] * (r & 1 ? inv * 0.0625f : inv);
                attend_store4(type, a.out, to_row + 32 * i + 8 * c + 4 * hf, v[0], v[1], v[2], v[3]);
            }
        if (hf == 0) attend_lse(a, sp.lse2, out_row, none ? -INFINITY : ref - kBias + log2_fast(sum));
    } else {
        const int64_t row = (((int64_t)split * tiles.live + place) * a.c.heads + head) * S::ROWS + (use - r0);
        if (hf == 0) sp.many_stats[row] = make_float2(ref == -INFINITY ? ref : ref - kBias, sum);
        if (none) return;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c)
                *reinterpret_cast<float4 *>(sp.many_sums + row * D + 32 * i + 8 * c + 4 * hf) =
                    make_float4(o[i][4 * c] * down, o[i][4 * c + 1] * (down * 0.0625f), o[i][4 * c + 2] * down,
                                o[i][4 * c + 3] * (down * 0.0625f));
    }
}

template <int KP, int PIECES, int D>
hipError_t launch(int type, const AttendArgs &a, const Splits &sp, int64_t workgroups, hipStream_t s) {
    using S = Shape<KP, PIECES, D>;
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t e = ensure_lds_bytes((const void *)k_attend_rows<KP, PIECES, D>, S::ALL, lds_set);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((k_attend_rows<KP, PIECES, D>), dim3((unsigned)workgroups), dim3(S::THREADS), S::ALL, s, a, sp, type);
    return hipGetLastError();
}
template <int KP, int PIECES>
hipError_t launch_for(int type, const AttendArgs &a, const Splits &sp, int64_t workgroups, hipStream_t s) {
    switch (a.c.D) {
        case 64: return launch<KP, PIECES, 64>(type, a, sp, workgroups, s);
        case 96: return launch<KP, PIECES, 96>(type, a, sp, workgroups, s);
        case 128: return launch<KP, PIECES, 128>(type, a, sp, workgroups, s);
    }
    if constexpr (PIECES == 1) return launch<KP, 1, 192>(type, a, sp, workgroups, s);
    return hipErrorInvalidValue;  // attend_rows_has
}

}  // namespace

hipError_t launch_attend_rows(int type, const AttendArgs &a, const Splits &sp, int64_t workgroups, hipStream_t s) {
    if (type == 0) return launch_for<2, 2>(type, a, sp, workgroups, s);
    const bool exact = type == 1 || a.lse != nullptr || a.mass != nullptr;
    return exact ? launch_for<2, 1>(type, a, sp, workgroups, s) : launch_for<1, 1>(type, a, sp, workgroups, s);
}

}  // namespace qmm
