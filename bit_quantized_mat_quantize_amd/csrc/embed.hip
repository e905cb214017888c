// embed.hip -- rows of a packed weight table by token id, decoded to fp32
// (gfx950): out[t][k] = scale * deq(W)[ids[t]][k].
//
// The decode is that of the weight formats (include/qmm.h): Q4_0 d*(q - 8),
// Q4_K and Q2_K (d*s_j)*q - dmin*m_j, Q6_K (d*s_j)*q.  In fp32 the products
// d*s_j*q and dmin*m_j are exact (11 bits of d, at most 7 of a scale and 6 of a
// code), so a value is rounded once by the subtraction, where there is one, and
// once by the scale.
//
// One thread decodes quads of four consecutive elements: a wavefront stores
// 1 KiB of a row with one 16-byte store per lane, and reads the 128 (Q4) to
// 256 bytes of codes behind it; the block's scales come from the same cache
// lines for all lanes.  The stores are most of the traffic (4 bytes per element
// against 0.33 to 0.82 read), so the kernel is bound by them for long inputs
// and by launch latency for single tokens.
#include "qmm_device.h"
#include "qmm_launch.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;

enum { F_Q4_0 = 0, F_Q4_K = 1, F_Q6_K = 2, F_Q2_K = 3 };

// four bytes at an address that is 2-byte (canonical Q4_0 and Q6_K blocks) or
// 4-byte aligned
template <bool ALIGN4>
__device__ __forceinline__ uint32_t ld4(const uint8_t *p) {
    if constexpr (ALIGN4) return *reinterpret_cast<const uint32_t *>(p);
    return ld_u16(p) | (ld_u16(p + 2) << 16);
}

// elements i .. i + 3 (i a multiple of 4) of block b of a table of NB blocks
// whose first section has dsec bytes (repacked layout)
template <int FMT, bool REP>
__device__ __forceinline__ float4 decode_quad(const uint8_t *__restrict__ w, int64_t NB, int64_t dsec, int64_t b,
                                              int i) {
    float v[4];
    if constexpr (FMT == F_Q4_0) {
        const uint8_t *head = REP ? w + 2 * b : w + b * kQ4_0Bytes;
        const uint8_t *qs = REP ? w + dsec + 16 * b : w + b * kQ4_0Bytes + 2;
        const uint32_t q = (ld4<REP>(qs + (i & 15)) >> ((i >> 4) * 4)) & 0x0f0f0f0fu;
        const float d = f16_bits_to_f32(ld_u16(head));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = d * (float)((int)((q >> (8 * e)) & 255u) - 8);
    } else if constexpr (FMT == F_Q4_K) {
        const uint8_t *head = REP ? w + 16 * b : w + b * kQ4_KBytes;
        const uint8_t *qs = REP ? w + 16 * NB + 128 * b : head + 16;
        const int j = i >> 5;
        const uint32_t q = (ld4<true>(qs + 32 * (j >> 1) + (i & 31)) >> ((j & 1) * 4)) & 0x0f0f0f0fu;
        const uint4 h = ld16(head);
        const Q4KScales r = unpack_scales(h.y, h.z, h.w);
        const int sh = 8 * (j & 3);
        const float ds = f16_bits_to_f32(h.x & 0xffffu) * (float)(((j & 4 ? r.s_hi : r.s_lo) >> sh) & 255u);
        const float dm = f16_bits_to_f32(h.x >> 16) * (float)(((j & 4 ? r.m_hi : r.m_lo) >> sh) & 255u);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ds * (float)((q >> (8 * e)) & 255u) - dm;
    } else if constexpr (FMT == F_Q6_K) {
        const uint8_t *blk = w + b * 210;  // canonical
        const uint8_t *head = REP ? w + 2 * b : blk + 208;
        const uint8_t *sc = REP ? w + dsec + 16 * b : blk + 192;
        const uint8_t *ql = REP ? w + dsec + 16 * NB + 128 * b : blk;
        const uint8_t *qh = REP ? w + dsec + 144 * NB + 64 * b : blk + 128;
        const int g = i >> 6, r = i & 63;
        const uint32_t lo = (ld4<REP>(ql + 32 * g + (r & 31)) >> ((r >> 5) * 4)) & 0x0f0f0f0fu;
        const uint32_t hi = (ld4<REP>(qh + r) >> (2 * g)) & 0x03030303u;
        const uint32_t u = lo | (hi << 4);
        const float ds = f16_bits_to_f32(ld_u16(head)) * (float)(int8_t)sc[i >> 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ds * (float)((int)((u >> (8 * e)) & 255u) - 32);
    } else {
        const uint8_t *blk = w + b * 84;  // canonical
        const uint32_t dd = ld4<true>(REP ? w + 4 * b : blk + 80);
        const uint8_t sc = (REP ? w + dsec + 16 * b : blk)[i >> 4];
        const uint8_t *qs = REP ? w + dsec + 16 * NB + 64 * b : blk + 16;
        const uint32_t q = (ld4<true>(qs + 32 * (i >> 7) + (i & 31)) >> (2 * ((i >> 5) & 3))) & 0x03030303u;
        const float ds = f16_bits_to_f32(dd & 0xffffu) * (float)(sc & 15);
        const float dm = f16_bits_to_f32(dd >> 16) * (float)(sc >> 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = ds * (float)((q >> (8 * e)) & 255u) - dm;
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// Work item = kThreads * quads<LONG> quads of one row; `chunks` items per row.  An
// id outside [0, N) gives a row of NaN and reads nothing of the table.  LONG: an
// output of more than the L2 caches hold goes past the caches, two quads per thread.
// 4099 rows of 8192 (134 MB, 4 buffers in turn) take 22.3 us so, 6.9 TB/s read and
// written, against 36.5 us with plain stores (Q4_K; 23.4 us with four quads); 2048 rows
// of 4096 (34 MB) 8.6 against 10.0 us.  Together with the quantization that reads the
// output (Q4_K, K = 8192, 5 buffers in turn): 34 MiB 21.5 against 21.7 us, 67 MiB 35.4
// against 35.5, 130 MiB 60 against 71.  Into a buffer that the 256 MB cache behind the L2
// still holds from the call before, plain stores are faster up to 145 MiB (34 MiB:
// 27.8 against 21.4 us for both kernels).
typedef float v4f __attribute__((ext_vector_type(4)));
template <bool LONG>
constexpr int quads = LONG ? 2 : 1;

template <int FMT, bool REP, bool LONG>
__global__ __launch_bounds__(kThreads) void k_embed_rows(const uint8_t *__restrict__ w, int64_t NB, int64_t dsec,
                                                         const int32_t *__restrict__ ids, int64_t items, int chunks,
                                                         float scale, float *__restrict__ out, int64_t N, int K) {
    constexpr int QK = FMT == F_Q4_0 ? QK4_0 : QK_K;
    constexpr int QPT = quads<LONG>;
    const int nb = K / QK;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t t = it / chunks;
        const int e0 = ((int)(it - t * chunks) * kThreads * QPT + threadIdx.x) * 4;
        const int64_t id = ids[t];
        const bool valid = id >= 0 && id < N;
        float4 v[QPT];
#pragma unroll
        for (int p = 0; p < QPT; ++p) {
            const int e = e0 + p * kThreads * 4;
            if (!valid) {
                const float nan = __builtin_nanf("");
                v[p] = make_float4(nan, nan, nan, nan);
            } else if (e < K) {
                v[p] = decode_quad<FMT, REP>(w, NB, dsec, id * nb + e / QK, e % QK);
            }
        }
#pragma unroll
        for (int p = 0; p < QPT; ++p) {
            const int e = e0 + p * kThreads * 4;
            const v4f o{v[p].x * scale, v[p].y * scale, v[p].z * scale, v[p].w * scale};
            v4f *to = reinterpret_cast<v4f *>(out + t * K + e);
            if (e < K && LONG) __builtin_nontemporal_store(o, to);
            else if (e < K) *to = o;
        }
    }
}

template <int FMT, bool REP, bool LONG>
hipError_t launch(const uint8_t *w, int64_t NB, int64_t dsec, const int32_t *ids, int64_t T, float scale, float *out,
                  int64_t N, int64_t K, hipStream_t s) {
    constexpr int per = kThreads * quads<LONG>;
    const int64_t chunks = (K / 4 + per - 1) / per;
    const int64_t items = T * chunks;
    const int64_t grid = items < (1 << 22) ? items : (1 << 22);  // 2^30 threads; the kernel strides over the rest
    hipLaunchKernelGGL((k_embed_rows<FMT, REP, LONG>), dim3((unsigned)grid), dim3(kThreads), 0, s, w, NB, dsec, ids,
                       items, (int)chunks, scale, out, N, (int)K);
    return hipGetLastError();
}

constexpr int64_t kLongBytes = 32 << 20;  // the L2 caches: 4 MiB for each of 8 XCDs
bool long_output(int64_t T, int64_t K) { return T * K * (int64_t)sizeof(float) >= kLongBytes; }

template <int FMT>
hipError_t launch_for(const uint8_t *w, bool repacked, int64_t NB, int64_t dsec, const int32_t *ids, int64_t T,
                      float scale, float *out, int64_t N, int64_t K, hipStream_t s) {
    const auto f = long_output(T, K) ? (repacked ? launch<FMT, true, true> : launch<FMT, false, true>)
                                     : (repacked ? launch<FMT, true, false> : launch<FMT, false, false>);
    return f(w, NB, dsec, ids, T, scale, out, N, K, s);
}

}  // namespace

bool embed_rows_long(int64_t T, int64_t K) { return long_output(T, K); }

hipError_t launch_embed_rows(int fmt, const uint8_t *w, bool repacked, const int32_t *ids, int64_t T, float scale,
                             float *out, int64_t N, int64_t K, hipStream_t s) {
    const int64_t NB = N * (K / (fmt == F_Q4_0 ? QK4_0 : QK_K));
    const int64_t dsec = ((fmt == F_Q2_K ? 4 : 2) * NB + 255) / 256 * 256;  // not used by Q4_K
    switch (fmt) {
        case F_Q4_0: return launch_for<F_Q4_0>(w, repacked, NB, dsec, ids, T, scale, out, N, K, s);
        case F_Q4_K: return launch_for<F_Q4_K>(w, repacked, NB, dsec, ids, T, scale, out, N, K, s);
        case F_Q6_K: return launch_for<F_Q6_K>(w, repacked, NB, dsec, ids, T, scale, out, N, K, s);
        default: return launch_for<F_Q2_K>(w, repacked, NB, dsec, ids, T, scale, out, N, K, s);
    }
}

}  // namespace qmm
