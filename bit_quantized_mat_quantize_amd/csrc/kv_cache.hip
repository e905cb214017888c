// kv_cache.hip -- rows of keys and values into the paged 4-bit cache, and entries
// back as numbers (gfx950).
//
// A block is 32 consecutive elements of a head under the rule of the Q4_0 encoder:
// d = -x/8 with x the element of largest magnitude (the first of equals), q =
// clamp(rint(x * (1/d)) + 8, 0, 15), values f16(d) * (q - 8).  A block that holds an
// infinity or NaN, or whose d passes fp16's range, gets d = NaN; where f16(d) is 0 all
// codes are 8.
//
// One thread holds eight elements, which are one 32-bit word of the cache; the four
// lanes of a block exchange their largest elements by DPP.  Keys and values of a row
// are one run of words, so the row's reads are whole and both sides run in one
// launch.  HBM bounds long prompts (4 or 2 bytes read per 9/16 written), the launch
// a decode step (61 rows: 3.4 us to write, 2.9 to read).
#include "kv_device.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;

// (|x|, x) of the block's element of largest magnitude, the first of equals; `bad`: any not finite
__device__ __forceinline__ void block_top(float &a, float &x, int &bad) {
#pragma unroll
    for (int step = 0; step < 2; ++step) {
        const float pa = step ? dpp_f32<0x4E>(a) : dpp_f32<0xB1>(a), px = step ? dpp_f32<0x4E>(x) : dpp_f32<0xB1>(x);
        bad |= step ? dpp_i32<0x4E>(bad) : dpp_i32<0xB1>(bad);
        const bool mine_first = ((threadIdx.x >> step) & 1) == 0;
        if (pa > a || (pa == a && !mine_first)) a = pa, x = px;
    }
}

// Rows per workgroup: their reads are on their way together, and the words of one group
// of four values, which share cache lines, come together.
template <int TYPE, int ROWS>
__global__ __launch_bounds__(kThreads) void k_cache_write(KvCache c, const void *__restrict__ k, int64_t ld_k,
                                                          const void *__restrict__ v, int64_t ld_v) {
    __shared__ int2 place[ROWS];
    const int words = c.heads * (c.D / 8);  // of a row's keys
    const int u = blockIdx.y * kThreads + threadIdx.x;
    const bool active = u < 2 * words;
    const int part = u >= words, e = active ? (part ? u - words : u) : 0;
    const int head = e / (c.D / 8), w = e - head * (c.D / 8);
    const void *src = part ? v : k;
    const int64_t ld = part ? ld_v : ld_k;
    const int r0 = blockIdx.x * ROWS;
    float x[ROWS][8];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[i][j] = 0.0f;
        if (active && r0 + i < c.T) kv_load8<TYPE>(src, (r0 + i) * ld + (int64_t)e * 8, x[i]);
    }
    kv_places<ROWS>(c, r0, place);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        float top = -1.0f, a = 0.0f;
        int bad = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[i][j]);
            if (m > top) top = m, a = x[i][j];
            bad |= !(m <= 3.402823466e38f);
        }
        block_top(top, a, bad);
        const float d = 0.0f - a / 8.0f;
        uint32_t h = f32_to_f16_bits(d);
        if (bad || (h & 0x7c00u) == 0x7c00u) h = 0x7e00u;
        const float id = (h & 0x7fffu) == 0 || h == 0x7e00u ? 0.0f : 1.0f / d;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float q = fminf(fmaxf(rintf((bad ? 0.0f : x[i][j]) * id) + 8.0f, 0.0f), 15.0f);
            word |= (uint32_t)q << (4 * j);
        }
        const int2 at = place[i];
        if (!active || at.x < 0) continue;
        uint8_t *to = kv_chunk(c, at.x, part, head);
        reinterpret_cast<uint32_t *>(to)[part ? kv_value_word(c.D, at.y, w) : kv_key_word(c.D, at.y, w)] = word;
        if ((w & 3) == 0) reinterpret_cast<uint16_t *>(to)[kv_scale_at(c, at.y, w >> 2)] = (uint16_t)h;
    }
}

// A thread stores 16 bytes, so that a wavefront stores whole lines: eight numbers of 16 bits, or four of a word's in fp32
// (two stores each of eight: 8192 rows of 8 heads of 128 29 us against 14).
template <int TYPE>
constexpr int kRead = TYPE == 0 ? 4 : 8;

template <int TYPE, int ROWS, bool PAST>
__global__ __launch_bounds__(kThreads) void k_cache_read(KvCache c, void *__restrict__ k, void *__restrict__ v) {
    constexpr int E = kRead<TYPE>;
    __shared__ int2 place[ROWS];
    const int units = c.heads * (c.D / E);
    const int u = blockIdx.y * kThreads + threadIdx.x, r0 = blockIdx.x * ROWS;
    kv_places<ROWS>(c, r0, place);
    if (u >= 2 * units) return;
    const int part = u >= units, e = part ? u - units : u, head = e / (c.D / E), at_head = e - head * (c.D / E);
    const int w = at_head * E / 8, first = at_head * E % 8;  // word; of its eight numbers
    uint32_t q[ROWS], d[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int2 at = place[i];
        q[i] = 0;
        d[i] = 0x7e00u;  // an entry that is not there is NaN
        if (at.x < 0) continue;
        const uint8_t *from = kv_chunk(c, at.x, part, head);
        q[i] = reinterpret_cast<const uint32_t *>(from)[part ? kv_value_word(c.D, at.y, w) : kv_key_word(c.D, at.y, w)];
        d[i] = reinterpret_cast<const uint16_t *>(from)[kv_scale_at(c, at.y, w >> 2)];
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (place[i].x == -2) continue;
        const float s = f16_bits_to_f32(d[i]);
        float x[E];
#pragma unroll
        for (int j = 0; j < E; ++j) x[j] = s * (float)((int)((q[i] >> (4 * (first + j))) & 15u) - 8);
        kv_store16<TYPE, PAST>(part ? v : k, ((int64_t)(r0 + i) * units + e) * E, x);
    }
}

// Eight rows a workgroup once that leaves enough workgroups for each CU: four to write, two to read.  8 heads of 128, us
// with eight against one: bf16, 2561 rows written in 10.2 and 8.8, 8192 in 16.7 and 19.9, 60013 in 102 and 112 (3.1
// TB/s); 4200 rows read in 9.0 and 8.9, 5000 in 9.3 and 9.8, 8000 in 11.7 and 14.3; fp32, 2100 rows read in 8.3 and
// 7.9, 3775 in 10.4 and 12.1.
bool eight_written(const KvCache &c, unsigned y) { return (int64_t)c.T * y >= 8 * 4 * 256; }
bool eight_read(const KvCache &c, unsigned y) { return (int64_t)c.T * y >= 8 * 2 * 256; }
// The L2 caches, 4 MiB for each of 8 XCDs: longer outputs go past them (us past and into them: bf16, 8192 rows 10.4 and
// 12.2, 20011 20.9 and 21.7, 80000 66 and 93; fp32, 8192 rows 15.0 and 16.7, 40000 63.5 and 85.9, 5.8 TB/s).
constexpr int64_t kLongBytes = 32 << 20;

template <int TYPE, int ROWS>
hipError_t launch_write_rows(const KvCache &c, const void *k, int64_t ld_k, const void *v, int64_t ld_v, unsigned y,
                             hipStream_t s) {
    hipLaunchKernelGGL((k_cache_write<TYPE, ROWS>), dim3((unsigned)((c.T + ROWS - 1) / ROWS), y), dim3(kThreads), 0, s, c, k,
                       ld_k, v, ld_v);
    return hipGetLastError();
}
template <int TYPE>
hipError_t launch_write(const KvCache &c, const void *k, int64_t ld_k, const void *v, int64_t ld_v, hipStream_t s) {
    const unsigned y = (unsigned)((2 * c.heads * (c.D / 8) + kThreads - 1) / kThreads);
    return eight_written(c, y) ? launch_write_rows<TYPE, 8>(c, k, ld_k, v, ld_v, y, s)
                            : launch_write_rows<TYPE, 1>(c, k, ld_k, v, ld_v, y, s);
}
template <int TYPE, int ROWS, bool PAST>
hipError_t launch_read_rows(const KvCache &c, void *k, void *v, unsigned y, hipStream_t s) {
    hipLaunchKernelGGL((k_cache_read<TYPE, ROWS, PAST>), dim3((unsigned)((c.T + ROWS - 1) / ROWS), y), dim3(kThreads), 0, s, c,
                       k, v);
    return hipGetLastError();
}
template <int TYPE>
hipError_t launch_read(const KvCache &c, void *k, void *v, hipStream_t s) {
    const unsigned y = (unsigned)((2 * c.heads * (c.D / kRead<TYPE>) + kThreads - 1) / kThreads);
    const bool past = (int64_t)c.T * c.heads * c.D * 2 * (TYPE == 0 ? 4 : 2) >= kLongBytes;
    if (!eight_read(c, y)) return launch_read_rows<TYPE, 1, false>(c, k, v, y, s);
    return past ? launch_read_rows<TYPE, 8, true>(c, k, v, y, s) : launch_read_rows<TYPE, 8, false>(c, k, v, y, s);
}

}  // namespace

hipError_t launch_cache_write(int type, const KvCache &c, const void *k, int64_t ld_k, const void *v, int64_t ld_v,
                              hipStream_t s) {
    if (type == 0) return launch_write<0>(c, k, ld_k, v, ld_v, s);
    return type == 1 ? launch_write<1>(c, k, ld_k, v, ld_v, s) : launch_write<2>(c, k, ld_k, v, ld_v, s);
}

hipError_t launch_cache_read(int type, const KvCache &c, void *k, void *v, hipStream_t s) {
    if (type == 0) return launch_read<0>(c, k, v, s);
    return type == 1 ? launch_read<1>(c, k, v, s) : launch_read<2>(c, k, v, s);
}

}  // namespace qmm
