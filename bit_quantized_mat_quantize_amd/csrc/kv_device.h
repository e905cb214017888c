// kv_device.h -- what the kernels of the 4-bit key/value cache share (gfx950):
// the cache's layout (include/qmm.h), the rows of ragged batches and the codes.
#pragma once

#include "qmm_device.h"
#include "qmm_launch.h"

namespace qmm {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ h2 as_h2(uint32_t u) { return __builtin_bit_cast(h2, u); }
__device__ __forceinline__ uint32_t as_u32(h2 h) { return __builtin_bit_cast(uint32_t, h); }

// ---- addresses.  A (page, keys or values, head) chunk holds the codes of `page`
// entries, D/2 bytes each, then their block scales as fp16 [D/32][page].
__device__ __forceinline__ int64_t kv_chunk_bytes(const KvCache &c) { return ((int64_t)c.D * 9 / 16) << c.page_log2; }
__device__ __forceinline__ uint8_t *kv_chunk(const KvCache &c, int64_t page, int part, int head) {
    return c.data + ((page * 2 + part) * c.heads + head) * kv_chunk_bytes(c);
}
// the 32-bit word of an entry t (within its page) that holds elements 8w .. 8w + 7
__device__ __forceinline__ int kv_key_word(int D, int t, int w) { return t * (D / 8) + (w & 3) * (D / 32) + (w >> 2); }
__device__ __forceinline__ int kv_value_word(int D, int t, int w) { return ((t >> 2) * (D / 8) + w) * 4 + (t & 3); }
// the fp16 scale of block b of entry t, counted from the chunk's start
__device__ __forceinline__ int kv_scale_at(const KvCache &c, int t, int b) {
    return ((c.D / 4) << c.page_log2) + (b << c.page_log2) + t;
}

// ---- rows.  Sequence b has the rows first .. first + count of the batch; its length
// counts them: row i stands at position len - count + i.  What the device arrays
// say is held within the batch and the table, whatever they hold.
struct KvRows {
    int first, count, len;
};
__device__ __forceinline__ KvRows kv_rows(const KvCache &c, int b) {
    KvRows r;
    if (c.starts == nullptr) {
        r.first = b;
        r.count = 1;
    } else {
        const int t0 = c.starts[b], t1 = c.starts[b + 1];
        r.first = t0 < 0 ? 0 : (t0 > c.T ? c.T : t0);
        const int end = t1 < r.first ? r.first : (t1 > c.T ? c.T : t1);
        r.count = end - r.first;
    }
    const int most = c.width << c.page_log2, len = c.lens[b];
    r.len = len < 0 ? 0 : (len > most ? most : len);
    return r;
}

// The last b < B with key(b) <= x for an ascending key, or -1; by the whole wavefront, 64
// candidates at a time (one dependent load for up to 64 sequences, two for 4096).
template <typename Key>
__device__ __forceinline__ int kv_last_not_above(int B, int64_t x, Key key) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = B;
    for (;;) {
        const int step = (n + 63) >> 6, at = lo + lane * step;
        const bool le = lane * step < n && key(at) <= x;
        const int c = __popcll(__ballot(le));
        if (c == 0) return -1;
        const int past = (c - 1) * step;
        lo += past;
        n = n - past < step ? n - past : step;
        if (step == 1) return lo;
    }
}

// the page that holds position pos of sequence b, or -1
__device__ __forceinline__ int kv_page(const KvCache &c, int b, int pos) {
    const int p = c.table[(int64_t)b * c.width + (pos >> c.page_log2)];
    return p >= 0 && p < c.pages ? p : -1;
}

// Where the rows r0 .. r0 + R - 1 of the batch are, for the whole workgroup: the page, or -1
// where that is not in the pool or the position is below 0, or -2 for a row of no
// sequence; and the entry of the page.  One search, then a lane per row: from the first row's
// sequence in doubling steps and back in halving ones, which is one read where the next sequence's rows
// lie behind, and 32 at most however many sequences have none (8196 rows of 8 heads of 128 in bf16, two of 65536
// sequences: written in 18.6 us, read in 11.5; a sequence at a time 4280 and 3730; a table of the two 17.9 and 10.7).
template <int R>
__device__ __forceinline__ void kv_places(const KvCache &c, int r0, int2 (&place)[R]) {
    static_assert(R <= 64, "one lane per row");
    if (threadIdx.x < 64) {
        int b = r0;
        if (c.starts != nullptr) b = kv_last_not_above(c.B, r0, [&](int i) { return (int64_t)c.starts[i]; });
        if (threadIdx.x < R) {
            const int r = r0 + threadIdx.x;
            if (c.starts == nullptr) b = r;
            else {
                if (b < 0) b = 0;  // rows before the first sequence: those behind may be its
                int step = 1;
                for (; b + step < c.B && c.starts[b + step] <= r; step *= 2) b += step;
                while ((step >>= 1) > 0)
                    if (b + step < c.B && c.starts[b + step] <= r) b += step;
            }
            int2 p = make_int2(-2, 0);
            if (r < c.T) {
                const KvRows k = kv_rows(c, b);
                if (r >= k.first && r < k.first + k.count) {
                    const int pos = k.len - k.count + (r - k.first);
                    p.x = pos >= 0 ? kv_page(c, b, pos) : -1;
                    p.y = pos & ((1 << c.page_log2) - 1);
                }
            }
            place[threadIdx.x] = p;
        }
    }
    __syncthreads();
}

// ---- element types: eight consecutive elements at a 16-byte aligned address
template <int TYPE>  // qmm_float_type
__device__ __forceinline__ void kv_load8(const void *base, int64_t at, float *v) {
    if constexpr (TYPE == 0) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 u = ld16(static_cast<const uint16_t *>(base) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (TYPE == 1) {
                v[2 * i] = f16_bits_to_f32(w[i] & 0xffffu);
                v[2 * i + 1] = f16_bits_to_f32(w[i] >> 16);
            } else {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
}
__device__ __forceinline__ void kv_load8(int type, const void *base, int64_t at, float *v) {
    if (type == 0) kv_load8<0>(base, at, v);
    else if (type == 1) kv_load8<1>(base, at, v);
    else kv_load8<2>(base, at, v);
}

// fp32 to bf16, to nearest even; NaN stays one
__device__ __forceinline__ uint32_t bf16_bits(float f) {
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}
// Four fp32 or eight 16-bit elements.  PAST: past the caches, for outputs that they cannot hold.
template <int TYPE, bool PAST>
__device__ __forceinline__ void kv_store16(void *base, int64_t at, const float *v) {
    if constexpr (TYPE == 0) {
        const f4 a = {v[0], v[1], v[2], v[3]};
        f4 *p = reinterpret_cast<f4 *>(static_cast<float *>(base) + at);
        if constexpr (PAST) __builtin_nontemporal_store(a, p);
        else *p = a;
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = TYPE == 1 ? f32_to_f16_bits(v[2 * i]) | (f32_to_f16_bits(v[2 * i + 1]) << 16)
                             : bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
        u32x4 *p = reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(base) + at);
        const u32x4 u = {w[0], w[1], w[2], w[3]};
        if constexpr (PAST) __builtin_nontemporal_store(u, p);
        else *p = u;
    }
}
template <int TYPE>
__device__ __forceinline__ void kv_store8(void *base, int64_t at, const float *v) {
    kv_store16<TYPE, false>(base, at, v);
    if constexpr (TYPE == 0) kv_store16<TYPE, false>(base, at + 4, v + 4);
}
__device__ __forceinline__ void kv_store8(int type, void *base, int64_t at, const float *v) {
    if (type == 0) kv_store8<0>(base, at, v);
    else if (type == 1) kv_store8<1>(base, at, v);
    else kv_store8<2>(base, at, v);
}

}  // namespace qmm
