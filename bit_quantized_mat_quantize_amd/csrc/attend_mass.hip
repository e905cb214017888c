// attend_mass.hip -- the weight that each entry of the cache got, for sequences of many
// query rows (gfx950): mass[j] += sum over rows and heads of the group of 2^(x - lse2),
// with the rows' lse2 from attention.hip and attend_rows.hip.
//
// A workgroup of four wavefronts owns 64 entries of a sequence and cache head and goes over
// all rows that see any of them, 64 at a time: two wavefronts take 32 entries each against
// the first 32 rows, the others the same entries against the others.  Two such workgroups
// share a compute unit, and one's products run beside the other's exponentials: 111 us at
// the size below; one workgroup of eight wavefronts took 121 with 128 entries and 126 with
// 128 rows.  The entries stay in registers, decoded to two fp16 pieces, whatever the queries are:
// weights are fp32 numbers.  The rows' queries come by direct loads into LDS, a step or two
// ahead, as the attention left them, fp16 and scaled: converting them anew in every
// workgroup took 180 us where loading them took 128 (three prompts of 700 rows, 28 heads of
// 128, fp32), and 121 with the rows' factors and lse loaded that way too.  Every entry's sum
// is formed in a fixed order: per lane over the rows, over the lanes, over the two
// wavefronts that share the entries.
#include "attend_device.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;

template <int PIECES, int D>
struct Shape {
    static constexpr int NB = D / 32, WORDS = D / 8;
    // wavefronts that share entries, each with 32 rows of a step; wavefronts with entries of their own
    static constexpr int STREAMS = 2, OWNERS = 2, ROWS = 32 * STREAMS, ENTRIES = 32 * OWNERS;
    static constexpr int PIECE = ROWS * D * 2, STAGE = PIECES * PIECE;  // bytes
    static constexpr int PER_PIECE = PIECE / 4096, LOADS = PIECES * PER_PIECE + 1;  // load instructions of a wavefront
    static constexpr int SLOTS = STAGE * 3 <= 75 * 1024 ? 3 : 2, BYTES = SLOTS * STAGE;
    static_assert(ROWS == 64 && BYTES <= 160 * 1024 - 8 * SLOTS * ROWS, "a lane loads a row's numbers; LDS of a compute unit");
};
// The place of 16-byte piece w of a row: eight lanes of one access meet eight of them, for rows of
// 128 bytes or multiples; rows of 192 bytes start 64 bytes apart already, four pieces are moved.
template <int D>
__device__ __forceinline__ int row_piece(int row, int w) {
    return row * D * 2 + ((D == 96 ? w ^ ((row >> 1) & 3) : w ^ (row & 7)) * 16);
}
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Query row r of a sequence as (token, head of the group), and steps of up to 64 rows without a
// division by the group g: x * ceil(2^21 / g) >> 21 is x / g for x < g + 64 and g <= 1024, because
// the quotient is too large by less than x / 2^21 < 1 / g.
struct Row {
    int token, head;
};
struct Steps {
    int group, magic;
    __device__ __forceinline__ explicit Steps(int g) : group(g), magic(((1 << 21) + g - 1) / g) {}
    __device__ __forceinline__ Row at(int r) const {
        const int t = r / group;
        return Row{t, r - t * group};
    }
    __device__ __forceinline__ Row on(const Row &r, int by) const {
        const int x = r.head + by, t = (int)(((uint32_t)x * (uint32_t)magic) >> 21);
        return Row{r.token + t, x - t * group};
    }
};

template <int PIECES, int D>
__global__ __launch_bounds__(kThreads, 2) void k_attend_mass_rows(AttendArgs a, Splits sp) {
    using S = Shape<PIECES, D>;
    constexpr int NB = S::NB, WORDS = S::WORDS;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ __attribute__((aligned(16))) float rows_at[S::SLOTS][2][S::ROWS];  // lse2 of a row; factor of its products
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, hf = lane >> 5;
    const int head = blockIdx.x % a.c.heads, x0 = blockIdx.x / a.c.heads;
    constexpr int ROWS = S::ROWS, OWNERS = S::OWNERS;
    const int tile = x0 / a.c.B, b = x0 - tile * a.c.B;  // more rows see earlier entries: first
    const int e0 = tile * S::ENTRIES, k0 = e0 + 32 * (wave % OWNERS), stream = wave / OWNERS;
    const KvRows rows = kv_rows(a.c, b);
    const int total = rows.count * a.group;
    if (total <= kMassRoom || e0 >= rows.len) return;
    // tokens that see any of the workgroup's entries
    const int before = rows.len - rows.count;
    int i0 = a.causal ? e0 - before : 0, i1 = a.window > 0 ? e0 + S::ENTRIES - 1 + a.window - before : rows.count;
    i0 = i0 < 0 ? 0 : i0;
    i1 = i1 > rows.count ? rows.count : i1;
    if (i0 >= i1) return;

    // ---- the entries: lane (n, hf) has words 2 i + hf of entry k0 + n
    h8 kh[2 * NB], kl[2 * NB];
    int shift;
    {
        Decode decode;
        decode.set();
        int at = k0 + n;
        const bool there = at < rows.len;
        at = there ? at : rows.len - 1;
        int page = kv_page(a.c, b, at);
        const bool nowhere = page < 0;
        page = nowhere ? 0 : page;
        const uint8_t *chunk = kv_chunk(a.c, page, 0, head);
        const int t = at & ((1 << a.c.page_log2) - 1);
        const uint32_t *row = reinterpret_cast<const uint32_t *>(chunk) + t * WORDS;
        uint32_t s[NB], top = 0;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            s[i] = nowhere ? 0x7e00u : reinterpret_cast<const uint16_t *>(chunk)[kv_scale_at(a.c, t, i)];
            if (!there) s[i] = 0;
            const uint32_t m = s[i] & 0x7fffu;
            top = m > top && m < 0x7c00u ? m : top;
        }
        shift = value_shift(wave_max_u16x2(top));
        const _Float16 unit = (_Float16)pow2i(shift);
#pragma unroll
        for (int i = 0; i < 2 * NB; ++i) {  // word 2 i + hf: block i / 2, word 2 (i % 2) + hf of it
            const uint32_t w = row[(2 * (i & 1) + hf) * NB + (i >> 1)], ss = s[i >> 1] | s[i >> 1] << 16;
            const h2 d = as_h2(ss) * h2{unit, unit};
            const h2 c[4] = {centred_even(decode.even(w)), centred_odd(decode.odd(w)), centred_even(decode.even(w >> 8)),
                             centred_odd(decode.odd(w >> 8))};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const h2 h = c[j] * d;
                kh[i][2 * j] = h.x, kh[i][2 * j + 1] = h.y;
                const h2 l = __builtin_elementwise_fma(c[j], d, -h);
                kl[i][2 * j] = l.x, kl[i][2 * j + 1] = l.y;
            }
        }
    }
    const float down = pow2i(-shift);

    // ---- rows into LDS: a wavefront loads a fourth of each piece, a lane the 16 bytes that belong to its place
    const uint32_t lds_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)lds);
    uint32_t place[S::PER_PIECE];
#pragma unroll
    for (int i = 0; i < S::PER_PIECE; ++i) {
        const int at = 1024 * (wave * S::PER_PIECE + i) + 16 * lane, row = at / (D * 2), w = at % (D * 2) / 16;
        place[i] = row * D * 2 + ((D == 96 ? w ^ ((row >> 1) & 3) : w ^ (row & 7)) * 16);
    }
    const int64_t row0 = attend_group_row(a, rows.first, head, 0);
    const uint32_t rows_lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) float *)&rows_at[0][0][0]);
    const Steps by_group(a.group);
    auto load = [&](int r0, int slot) {  // rows from r0 on: what lies behind the last of all is not read
#pragma unroll
        for (int k = 0; k < PIECES; ++k) {
            const uint64_t base = (uint64_t)(uintptr_t)(sp.queries + k * sp.query_piece + (row0 + r0) * D);
            const u32x4 r = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, (uint32_t)((total - r0 < ROWS ? total - r0 : ROWS) * D * 2),
                             0x00020000u};
#pragma unroll
            for (int i = 0; i < S::PER_PIECE; ++i)
                asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(
                                 lds_at + slot * S::STAGE + k * S::PIECE + 1024 * (wave * S::PER_PIECE + i)),
                             "v"(place[i]), "s"(r) : "m0", "memory");
        }
        // the wavefronts load the same by twos, so that all have as many loads
        const uint64_t base = (uint64_t)(uintptr_t)((wave & 1 ? sp.factors : sp.lse2) + row0 + r0);
        const u32x4 r = {(uint32_t)base, (uint32_t)(base >> 32) & 0xffffu, (uint32_t)((total - r0 < ROWS ? total - r0 : ROWS) * 4),
                         0x00020000u};
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(
                         rows_lds + slot * (8 * ROWS) + (wave & 1) * (4 * ROWS)),
                     "v"(4 * lane), "s"(r) : "m0", "memory");
    };
    float got[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) got[r] = 0.0f;
    const int begin = i0 * a.group, end = i1 * a.group;
    Row mine = by_group.on(by_group.at(begin), 32 * stream);
    constexpr int AHEAD = S::SLOTS - 1;
    for (int i = 0; i < AHEAD; ++i)
        if (begin + i * ROWS < end) load(begin + i * ROWS, i);
    int slot = 0;
    for (int r0 = begin; r0 < end; r0 += ROWS, slot = slot + 1 == S::SLOTS ? 0 : slot + 1) {
        // this wavefront's part of the step's rows is there, then everybody's; nobody reads the slot that is filled next
        if (AHEAD > 1 && r0 + ROWS < end) wait_loads<(AHEAD > 1 ? S::LOADS : 0)>();
        else wait_loads<0>();
        __syncthreads();
        if (r0 + AHEAD * ROWS < end) load(r0 + AHEAD * ROWS, slot == 0 ? S::SLOTS - 1 : slot - 1);
        const int wr0 = r0 + 32 * stream, wr1 = wr0 + 31;
        if (wr0 < end && k0 < rows.len) {
            int lo0, hi0, lo1, hi1;  // what the first and the last of the wavefront's rows see
            const int last = by_group.on(mine, 31).token;
            attend_span(a, rows, mine.token, lo0, hi0);
            attend_span(a, rows, last < rows.count ? last : rows.count - 1, lo1, hi1);
            if (k0 < hi1 && k0 + 32 > lo0) {
                const uint8_t *from = lds + slot * S::STAGE;
                f16v x;
#pragma unroll
                for (int r = 0; r < 16; ++r) x[r] = 0.0f;
#pragma unroll
                for (int i = 0; i < 2 * NB; ++i) {
                    const uint8_t *p = from + row_piece<D>(32 * stream + n, 2 * i + hf);
                    const h8 qh = *reinterpret_cast<const h8 *>(p);
                    x = mfma32(kh[i], qh, x);
                    if constexpr (PIECES == 2) {
                        const h8 ql = *reinterpret_cast<const h8 *>(p + S::PIECE);
                        x = mfma32(kh[i], ql, x);
                    }
                    x = mfma32(kl[i], qh, x);
                }
                // a row that has nothing weighs nothing
                const float lse = rows_at[slot][0][32 * stream + n], up = lse == -INFINITY ? lse : -lse;
                const float by = lse == -INFINITY ? 0.0f : rows_at[slot][1][32 * stream + n] * down;
                if (k0 < lo1 || k0 + 32 > hi0 || wr1 >= total) {
                    int lo = 1, hi = 0;
                    const int token = by_group.on(mine, n).token;
                    if (token < rows.count) attend_span(a, rows, token, lo, hi);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int at = k0 + 8 * (r >> 2) + 4 * hf + (r & 3);
                        got[r] += at >= lo && at < hi ? exp2_fast(fmaf(x[r], by, up)) : 0.0f;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) got[r] += exp2_fast(fmaf(x[r], by, up));
                }
            }
        }
        mine = by_group.on(mine, ROWS);
    }
    // over the 32 rows that lie along the lanes, then over the wavefronts that share the entries
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) got[r] += __shfl_xor(got[r], o, 64);
    __syncthreads();
    float *other = reinterpret_cast<float *>(lds);
    if (n == 0)
#pragma unroll
        for (int r = 0; r < 16; ++r) other[32 * wave + 8 * (r >> 2) + 4 * hf + (r & 3)] = got[r];
    __syncthreads();
    if (threadIdx.x < S::ENTRIES && e0 + (int)threadIdx.x < rows.len) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < S::STREAMS; ++i) sum += other[S::ENTRIES * i + threadIdx.x];
        a.mass[((int64_t)b * a.c.heads + head) * a.ld_mass + e0 + threadIdx.x] += sum;
    }
}

template <int PIECES, int D>
hipError_t launch(int type, const AttendArgs &a, const Splits &sp, hipStream_t s) {
    using S = Shape<PIECES, D>;
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t e = ensure_lds_bytes((const void *)k_attend_mass_rows<PIECES, D>, S::BYTES, lds_set);
    if (e != hipSuccess) return e;
    const int64_t tiles = (((int64_t)a.c.width << a.c.page_log2) + S::ENTRIES - 1) / S::ENTRIES;
    hipLaunchKernelGGL((k_attend_mass_rows<PIECES, D>), dim3((unsigned)(a.c.B * tiles * a.c.heads)), dim3(kThreads), S::BYTES, s, a, sp);
    return hipGetLastError();
}
template <int PIECES>
hipError_t launch_for(int type, const AttendArgs &a, const Splits &sp, hipStream_t s) {
    switch (a.c.D) {
        case 64: return launch<PIECES, 64>(type, a, sp, s);
        case 96: return launch<PIECES, 96>(type, a, sp, s);
        case 128: return launch<PIECES, 128>(type, a, sp, s);
        case 192: return launch<PIECES, 192>(type, a, sp, s);
        default: return launch<PIECES, 256>(type, a, sp, s);
    }
}

}  // namespace

hipError_t launch_attend_mass_rows(int type, const AttendArgs &a, const Splits &sp, hipStream_t s) {
    return type == 0 ? launch_for<2>(type, a, sp, s) : launch_for<1>(type, a, sp, s);
}

}  // namespace qmm
