// attend_mass.hip -- the weight that each entry of the cache got, for sequences of many
// query rows (gfx950): mass[j] += sum over rows and heads of the group of 2^(x - lse2),
// with the rows' lse2 from attend_rows.hip.
//
// A workgroup owns 128 entries of a sequence and cache head and goes over all rows that
// see any of them, 64 at a time: wavefronts 0 .. 3 take 32 entries each against the first
// 32 rows, 4 .. 7 the same entries against the others.  The entries stay in registers,
// decoded to fp16 (two pieces for fp32 queries, as in attend_rows.hip); the rows come through
// LDS, converted once for the workgroup.  Every entry's sum is formed in a fixed order
// by its owner: per lane over the rows, over the lanes, over the two halves.
#include "attend_device.h"

namespace qmm {
namespace {

constexpr int kThreads = 512, kRows = 64, kEntries = 128;

template <int PIECES, int D>
struct Shape {
    static constexpr int NB = D / 32, WORDS = D / 8;
    static constexpr int ROW = D == 96 ? 128 : D;  // elements of a row in LDS
    static constexpr int PIECE = kRows * ROW * 2, STAGE = PIECES * PIECE, BYTES = 2 * STAGE;
};
template <int D>
__device__ __forceinline__ int row_piece(int row, int w) {
    return row * (D == 96 ? 128 : D) * 2 + ((w ^ (row & 7)) * 16);
}

template <int PIECES, int D>
__global__ __launch_bounds__(kThreads, 1) void k_attend_mass_rows(AttendArgs a, Splits sp, int type, int tiles) {
    using S = Shape<PIECES, D>;
    constexpr int NB = S::NB, WORDS = S::WORDS;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float2 rows_at[2][kRows];  // factor of a row's products, -lse2
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31, hf = lane >> 5;
    const int head = blockIdx.x % a.c.heads, x0 = blockIdx.x / a.c.heads, b = x0 / tiles;
    const int e0 = (x0 - b * tiles) * kEntries, k0 = e0 + 32 * (wave & 3), stream = wave >> 2;
    const KvRows rows = kv_rows(a.c, b);
    const int total = rows.count * a.group;
    if (total <= sp.few_room || e0 >= rows.len) return;
    // tokens that see any of the 128 entries
    const int before = rows.len - rows.count;
    int i0 = a.causal ? e0 - before : 0, i1 = a.window > 0 ? e0 + kEntries - 1 + a.window - before : rows.count;
    i0 = i0 < 0 ? 0 : i0;
    i1 = i1 > rows.count ? rows.count : i1;
    if (i0 >= i1) return;

    // ---- the entries: lane (n, hf) has words 2 i + hf of entry k0 + n
    h8 kh[2 * NB], kl[PIECES == 2 ? 2 * NB : 1];
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
                if constexpr (PIECES == 2) {
                    const h2 l = __builtin_elementwise_fma(c[j], d, -h);
                    kl[i][2 * j] = l.x, kl[i][2 * j + 1] = l.y;
                }
            }
        }
    }
    const float down = pow2i(-shift);

    // ---- rows into LDS: eight threads a row, words tid % 8, + 8, ..
    constexpr int EACH = (WORDS + 7) / 8;
    const int sr = threadIdx.x >> 3, sw = threadIdx.x & 7;
    float f[EACH][8];
    float row_lse = 0.0f;
    auto load = [&](int r0) {
        int r = r0 + sr;
        const bool live = r < total;
        r = live ? r : total - 1;
        const int64_t out_row = attend_out_row(a, rows, head, r), at = attend_at(a, out_row, a.ld_q);
#pragma unroll
        for (int j = 0; j < EACH; ++j)
            if (sw + 8 * j < WORDS) kv_load8(type, a.q, at + 8 * (sw + 8 * j), f[j]);
        row_lse = live ? sp.lse2[out_row] : -INFINITY;
    };
    auto put = [&](int stage) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < EACH; ++j)
            if (sw + 8 * j < WORDS)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t u = __float_as_uint(f[j][e]) & 0x7fffffffu;
                    top = u > top ? u : top;
                }
        for (int o = 1; o < 8; o <<= 1) {
            const uint32_t u = __shfl_xor(top, o, 64);
            top = u > top ? u : top;
        }
        const int qs = query_shift(top);
        const float by = a.scale < 0.0f ? -pow2i(qs) : pow2i(qs);
        uint8_t *to = lds + stage * S::STAGE;
#pragma unroll
        for (int j = 0; j < EACH; ++j)
            if (sw + 8 * j < WORDS) {
                h8 hi, lo;
                query_pieces<PIECES>(f[j], by, hi, lo);
                *reinterpret_cast<h8 *>(to + row_piece<D>(sr, sw + 8 * j)) = hi;
                if constexpr (PIECES == 2) *reinterpret_cast<h8 *>(to + S::PIECE + row_piece<D>(sr, sw + 8 * j)) = lo;
            }
        // a row that has nothing (or is none) weighs nothing
        if (sw == 0)
            rows_at[stage][sr] = row_lse == -INFINITY ? make_float2(0.0f, -INFINITY)
                                                      : make_float2((top >> 23) == 255 ? __builtin_nanf("") : fabsf(a.scale) * pow2i(-qs), -row_lse);
    };

    float got[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) got[r] = 0.0f;
    const int first = i0 * a.group / kRows * kRows, end = i1 * a.group;
    load(first);
    put(0);
    for (int r0 = first, stage = 0; r0 < end; r0 += kRows, stage ^= 1) {
        __syncthreads();
        if (r0 + kRows < end) load(r0 + kRows);
        const int wr0 = r0 + 32 * stream, wr1 = wr0 + 31;
        if (wr0 < end && k0 < rows.len) {
            int lo0, hi0, lo1, hi1;  // what the first and the last of the wavefront's rows see
            attend_span(a, rows, wr0 / a.group, lo0, hi0);
            attend_span(a, rows, (wr1 < total ? wr1 : total - 1) / a.group, lo1, hi1);
            if (k0 < hi1 && k0 + 32 > lo0) {
                const uint8_t *from = lds + stage * S::STAGE;
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
                        x = mfma32(kl[i], qh, x);
                    }
                }
                const float2 row = rows_at[stage][32 * stream + n];
                const float by = row.x * down;
                if (k0 < lo1 || k0 + 32 > hi0 || wr1 >= total) {
                    int lo = 1, hi = 0;
                    if (wr0 + n < total) attend_span(a, rows, (wr0 + n) / a.group, lo, hi);
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int at = k0 + 8 * (r >> 2) + 4 * hf + (r & 3);
                        got[r] += at >= lo && at < hi ? exp2_fast(fmaf(x[r], by, row.y)) : 0.0f;
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 16; ++r) got[r] += exp2_fast(fmaf(x[r], by, row.y));
                }
            }
        }
        if (r0 + kRows < end) put(stage ^ 1);
    }
    // over the 32 rows that lie along the lanes, then over the two halves
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) got[r] += __shfl_xor(got[r], o, 64);
    __syncthreads();
    float *other = reinterpret_cast<float *>(lds);
    if (stream == 1 && n == 0)
#pragma unroll
        for (int r = 0; r < 16; ++r) other[32 * (wave & 3) + 8 * (r >> 2) + 4 * hf + (r & 3)] = got[r];
    __syncthreads();
    if (stream == 0 && n == 0) {
        float *mass = a.mass + ((int64_t)b * a.c.heads + head) * a.ld_mass;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const int e = 8 * (r >> 2) + 4 * hf + (r & 3);
            if (k0 + e < rows.len) mass[k0 + e] += got[r] + other[32 * wave + e];
        }
    }
}

template <int PIECES, int D>
hipError_t launch(int type, const AttendArgs &a, const Splits &sp, hipStream_t s) {
    using S = Shape<PIECES, D>;
    static std::atomic<uint64_t> lds_set{0};
    const hipError_t e = ensure_lds_bytes((const void *)k_attend_mass_rows<PIECES, D>, S::BYTES, lds_set);
    if (e != hipSuccess) return e;
    const int64_t tiles = attend_mass_tiles(a);
    hipLaunchKernelGGL((k_attend_mass_rows<PIECES, D>), dim3((unsigned)(a.c.B * tiles * a.c.heads)), dim3(kThreads), S::BYTES, s,
                       a, sp, type, (int)tiles);
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

int64_t attend_mass_tiles(const AttendArgs &a) {
    return (((int64_t)a.c.width << a.c.page_log2) + kEntries - 1) / kEntries;
}

hipError_t launch_attend_mass_rows(int type, const AttendArgs &a, const Splits &sp, hipStream_t s) {
    return type == 0 ? launch_for<2>(type, a, sp, s) : launch_for<1>(type, a, sp, s);
}

}  // namespace qmm
