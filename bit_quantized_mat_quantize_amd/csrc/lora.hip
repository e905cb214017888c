// lora.hip -- low-rank adapters of many requests on top of a shared projection
// (gfx950).  Row m of a batch asks for adapter e = ids[m]:
//
//     out[m][n] = base[m][n] + s_e * sum_{r < rank_e} B[e][n][r] * v[m][r],
//     v[m][r]   = sum_k A[e][r][k] * x[m][k]
//
// in two launches: k_lora_shrink computes v (a long contraction with few
// outputs: K is split over workgroups and their partial sums go to the
// workspace), k_lora_expand adds the partials in a fixed order, scales them and
// multiplies with B.
//
// Both work on tiles of 16 consecutive rows.  The rows of a tile may ask for
// different adapters in any order: a wavefront holds the tile's ids in its
// lanes, takes the distinct ones one after another (ballot), and stores the rows
// that match.  Rows of one request are neighbours in a prefill batch, so most
// tiles have one adapter and nothing is sorted; in a decode batch each row may
// have its own, and `zsplit` workgroups per tile take the distinct adapters
// z, z + zsplit, ... so that they run beside one another.
//
// The products run on the fp32 matrix instruction (v_mfma_f32_16x16x4_f32): x
// is fp32 and the result is, so x is not rounded to 16 bits, and A and B in
// fp16 or bf16 convert exactly.  Its rate (256 flop per cycle and CU) is above
// what these products need up to ranks of about 64, where x, base and out are
// what has to move.  A lane feeds four or eight consecutive k (or r) to
// consecutive instructions, with the same assignment on both operands: the sum
// over k does not mind the order, and every load is 8 to 32 contiguous bytes
// per lane, whole 64- or 128-byte pieces per row.
#include "qmm_device.h"
#include "qmm_launch.h"

namespace qmm {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTileRows = 16;
constexpr int kStep = 32;  // k per wavefront step of the shrink

// ---- element types: T is the storage type of A and B
struct BF16 {
    uint16_t b;
};
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(BF16 v) { return __uint_as_float((uint32_t)v.b << 16); }

// n consecutive elements at an address aligned to the whole load
template <typename T, int n>
__device__ __forceinline__ void load_n(const T *p, float (&v)[n]) {
    struct alignas(sizeof(T) * n < 16 ? sizeof(T) * n : 16) Pack {
        T e[n];
    };
    const Pack q = *reinterpret_cast<const Pack *>(p);
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = to_f32(q.e[i]);
}

__device__ __forceinline__ int rank_of(const int32_t *ranks, int e, int R) {
    if (ranks == nullptr) return R;
    const int r = ranks[e];
    return r < 0 ? 0 : (r > R ? R : r);
}

// The distinct adapters of a tile, one call of f(e, match) each; match has a bit
// for every row that asks for e.  Every wavefront of a workgroup sees the same
// ids, so f may hold barriers.
template <typename F>
__device__ __forceinline__ void for_each_adapter(int id, bool valid, int z, int zsplit, F f) {
    uint64_t rem = __ballot(valid);
    for (int n = 0; rem != 0; ++n) {
        const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
        const uint64_t match = __ballot(valid && id == e);
        rem &= ~match;
        if (n % zsplit == z) f(e, (uint32_t)match);
    }
}

// ---- v: partial sums P[s][m][r] over the k steps of split s.
// Workgroup = (tile, z, block of RT * 16 ranks, split); its wavefronts take the
// steps in turn and add their tiles in LDS.  Rows that do not match read the
// first matching row's x (same cache lines), ranks past the adapter's own read
// its last one; neither is used.
template <typename T, int RT>
__global__ __launch_bounds__(kThreads) void k_lora_shrink(const T *__restrict__ A, int64_t E, int R,
                                                          const int32_t *__restrict__ ranks,
                                                          const float *__restrict__ x,
                                                          const int32_t *__restrict__ ids, int64_t M, int K,
                                                          int splits, int rank_blocks, int zsplit, int Rp,
                                                          float *__restrict__ P) {
    __shared__ v4f red[kWaves][RT][kWave];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane & 15, g = lane >> 4;
    uint32_t b = blockIdx.x;
    const int s = (int)(b % splits);
    b /= splits;
    const int r0 = (int)(b % rank_blocks) * RT * 16;
    b /= rank_blocks;
    const int z = (int)(b % (uint32_t)zsplit);
    const int64_t m0 = (int64_t)(b / zsplit) * kTileRows;
    const int id = lane < kTileRows && m0 + lane < M ? ids[m0 + lane] : -1;
    const int steps = K / kStep, per = (steps + splits - 1) / splits;
    const int st0 = s * per, st1 = st0 + per < steps ? st0 + per : steps;

    for_each_adapter(id, id >= 0 && id < E, z, zsplit, [&](int e, uint32_t match) {
        const int rank = rank_of(ranks, e, R);
        if (rank <= r0) return;
        const int xr = match >> row & 1 ? row : __builtin_ctz(match);
        const float *xp = x + (m0 + xr) * K + 8 * g;
        const T *ap[RT];
        v4f acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = r0 + t * 16 + row;
            ap[t] = A + ((int64_t)e * R + (r < rank ? r : rank - 1)) * K + 8 * g;
            acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll 2
        for (int st = st0 + wave; st < st1; st += kWaves) {
            float xv[8];
            load_n<float, 8>(xp + st * kStep, xv);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                float av[8];
                load_n<T, 8>(ap[t] + st * kStep, av);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[i], av[i], acc[t], 0, 0, 0);
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) red[wave][t][lane] = acc[t];
        __syncthreads();
        for (int i = threadIdx.x; i < RT * kWave; i += kThreads) {
            const int t = i >> 6, l = i & 63;
            v4f v = red[0][t][l];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) v += red[w][t][l];
            const int r = r0 + t * 16 + (l & 15);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int mr = 4 * (l >> 4) + q;
                if (match >> mr & 1) P[((int64_t)s * M + m0 + mr) * Rp + r] = v[q];
            }
        }
        __syncthreads();
    });
}

// ---- out = base + v B^T.  Workgroup = (tile, z, strip of columns): the tile's v
// (partials added in order, scaled) goes to LDS once per adapter, then each
// wavefront multiplies 16 columns of B at a time: B's rows are the matrix
// instruction's rows, so a lane ends with four consecutive columns of one output
// row.  VEC: base and out rows are 16-byte aligned (16-byte accesses); BV: R is a
// multiple of 4 (B in loads of four elements).
template <typename T, bool VEC, bool BV, int NT>
__global__ __launch_bounds__(kThreads) void k_lora_expand(const T *__restrict__ B, int64_t E, int R,
                                                          const float *__restrict__ scales,
                                                          const int32_t *__restrict__ ranks,
                                                          const int32_t *__restrict__ ids, int64_t M,
                                                          const float *__restrict__ P, int splits, int Rp,
                                                          const float *base, int64_t ld_base, float *out,
                                                          int64_t ld_out, int64_t N, int strips, int zsplit) {
    extern __shared__ float vs[];  // [kTileRows][Rp + 4]
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row = lane & 15, g = lane >> 4;
    const int vld = Rp + 4;
    uint32_t b = blockIdx.x;
    const int64_t n_wave = (int64_t)(b % strips * kWaves + wave) * (16 * NT);
    b /= strips;
    const int z = (int)(b % (uint32_t)zsplit);
    const int64_t m0 = (int64_t)(b / zsplit) * kTileRows;
    const int64_t m = m0 + row;
    const int id = m < M ? ids[m] : -1;
    const bool valid = id >= 0 && id < E;

    // rows without an adapter: the base as it is; an id that names none: NaN
    if (z == 0 && m < M && !valid && !(id == -1 && base == out)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int64_t n = n_wave + 16 * t + 4 * g;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (n + q < N)
                    out[m * ld_out + n + q] = id == -1 ? base[m * ld_base + n + q] : __builtin_nanf("");
        }
    }

    for_each_adapter(id, valid && lane < kTileRows, z, zsplit, [&](int e, uint32_t match) {
        const int rank = rank_of(ranks, e, R);
        const float scale = scales != nullptr ? scales[e] : 1.0f;
        for (int i = threadIdx.x; i < kTileRows * Rp; i += kThreads) {
            const int mr = i / Rp, r = i - mr * Rp;
            float v = 0.f;
            if ((match >> mr & 1) && r < rank) {
                const float *p = P + (m0 + mr) * Rp + r;
                for (int s = 0; s < splits; ++s) v += p[(int64_t)s * M * Rp];
                v *= scale;
            }
            vs[mr * vld + r] = v;
        }
        __syncthreads();
        const bool mine = match >> row & 1;
        v4f acc[NT], bv[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
            const int64_t n = n_wave + 16 * t + 4 * g;
            bv[t] = v4f{0.f, 0.f, 0.f, 0.f};
            if (mine) {
                if (VEC && n + 3 < N) {
                    bv[t] = *reinterpret_cast<const v4f *>(base + m * ld_base + n);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n + q < N) bv[t][q] = base[m * ld_base + n + q];
                }
            }
        }
        for (int c = 0; c < rank; c += 16) {
            const int r = c + 4 * g;
            const v4f v = *reinterpret_cast<const v4f *>(vs + row * vld + r);
            float w[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int64_t n = n_wave + 16 * t + row;
                const T *p = B + ((int64_t)e * N + (n < N ? n : N - 1)) * R + r;
#pragma unroll
                for (int i = 0; i < 4; ++i) w[t][i] = 0.f;
                if (BV) {
                    if (r < rank) load_n<T, 4>(p, w[t]);
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[t][i] = r + i < rank ? w[t][i] : 0.f;
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (r + i < rank) w[t][i] = to_f32(p[i]);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(w[t][i], v[i], acc[t], 0, 0, 0);
        }
        if (mine) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int64_t n = n_wave + 16 * t + 4 * g;
                const v4f o = bv[t] + acc[t];
                if (VEC && n + 3 < N) {
                    *reinterpret_cast<v4f *>(out + m * ld_out + n) = o;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n + q < N) out[m * ld_out + n + q] = o[q];
                }
            }
        }
        __syncthreads();
    });
}

// ---- launch shapes (host only; they need no device)
constexpr int kTargetGroups = 1024;  // workgroups that fill the chip: four per CU
constexpr int kMaxSplits = 32;

struct Shape {
    int rt, rank_blocks, Rp, zsplit, splits;
    int64_t tiles;
};
Shape shape(int64_t M, int64_t R, int64_t K, int64_t E) {
    Shape h;
    h.rt = R <= 16 ? 1 : (R <= 32 ? 2 : 4);
    h.rank_blocks = (int)((R + 16 * h.rt - 1) / (16 * h.rt));
    h.Rp = h.rank_blocks * h.rt * 16;
    h.tiles = (M + kTileRows - 1) / kTileRows;
    h.zsplit = M <= 64 ? 16 : (M <= 512 ? 4 : 1);
    if (h.zsplit > E) h.zsplit = (int)E;
    if (h.zsplit > M) h.zsplit = (int)M;
    const int64_t groups = h.tiles * h.zsplit * h.rank_blocks;
    const int64_t most = (K / kStep + 2 * kWaves - 1) / (2 * kWaves);  // two steps for each wavefront at least
    int64_t s = (kTargetGroups + groups - 1) / groups;
    s = s > kMaxSplits ? kMaxSplits : s;
    h.splits = (int)(s > most ? most : s);
    return h;
}

template <typename T, int RT>
hipError_t shrink(const LoraArgs &a, const Shape &h, hipStream_t s) {
    const int64_t grid = h.tiles * h.zsplit * h.rank_blocks * h.splits;
    hipLaunchKernelGGL((k_lora_shrink<T, RT>), dim3((unsigned)grid), dim3(kThreads), 0, s,
                       static_cast<const T *>(a.A), a.E, (int)a.R, a.ranks, a.x, a.ids, a.M, (int)a.K, h.splits,
                       h.rank_blocks, h.zsplit, h.Rp, a.ws);
    return hipGetLastError();
}

constexpr int kNT = 4;
int64_t expand_strips(int64_t N) { return (N + kWaves * 16 * kNT - 1) / (kWaves * 16 * kNT); }

template <typename T, bool VEC, bool BV>
hipError_t expand(const LoraArgs &a, const Shape &h, hipStream_t s) {
    const int64_t strips = expand_strips(a.N);
    const size_t lds = sizeof(float) * kTileRows * (h.Rp + 4);
    hipLaunchKernelGGL((k_lora_expand<T, VEC, BV, kNT>), dim3((unsigned)(strips * h.zsplit * h.tiles)), dim3(kThreads),
                       lds, s, static_cast<const T *>(a.B), a.E, (int)a.R, a.scales, a.ranks, a.ids, a.M, a.ws,
                       h.splits, h.Rp, a.base, a.ld_base, a.out, a.ld_out, a.N, (int)strips, h.zsplit);
    return hipGetLastError();
}

template <typename T>
hipError_t both(const LoraArgs &a, hipStream_t s) {
    const Shape h = shape(a.M, a.R, a.K, a.E);
    hipError_t e = h.rt == 1 ? shrink<T, 1>(a, h, s) : (h.rt == 2 ? shrink<T, 2>(a, h, s) : shrink<T, 4>(a, h, s));
    if (e != hipSuccess) return e;
    const bool vec = a.ld_base % 4 == 0 && a.ld_out % 4 == 0, bv = a.R % 4 == 0;
    return vec ? (bv ? expand<T, true, true>(a, h, s) : expand<T, true, false>(a, h, s))
               : (bv ? expand<T, false, true>(a, h, s) : expand<T, false, false>(a, h, s));
}

}  // namespace

int64_t lora_workspace_bytes(int64_t M, int64_t R, int64_t K, int64_t E) {
    const Shape h = shape(M, R, K, E);
    return (int64_t)sizeof(float) * h.splits * M * h.Rp;
}

bool lora_grid_ok(int64_t M, int64_t N, int64_t R, int64_t K, int64_t E) {
    const Shape h = shape(M, R, K, E);
    const int64_t most = (int64_t(1) << 32) / kThreads - 1;  // threads of one launch are counted in 32 bits
    return h.tiles * h.zsplit * h.rank_blocks * h.splits <= most && expand_strips(N) * h.zsplit * h.tiles <= most;
}

hipError_t launch_lora_add(int type, const LoraArgs &a, hipStream_t s) {
    switch (type) {
        case 0: return both<float>(a, s);
        case 1: return both<_Float16>(a, s);
        default: return both<BF16>(a, s);
    }
}

}  // namespace qmm
