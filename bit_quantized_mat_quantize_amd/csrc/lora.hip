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
// have its own, and `zsplit` workgroups share a tile so that its adapters run
// beside one another.
//
// The first product runs on the fp32 matrix instruction (v_mfma_f32_16x16x4_f32): x
// is fp32 and the result is, so x is not rounded to 16 bits, and A in fp16 or bf16
// converts exactly.  Its rate (256 flop per cycle and CU) is above what the product
// needs up to ranks of about 64, where x is what has to move.  The second product
// has few k and many outputs: there a 16-bit B goes to the bf16 instruction, fp16 in
// two pieces, and v in three (Operand).  A lane feeds four or eight consecutive k (or r) to
// consecutive instructions, with the same assignment on both operands: the sum over
// k does not mind the order, and every load is 8 to 32 contiguous bytes per lane,
// whole 64- or 128-byte pieces per row.
#include "qmm_device.h"
#include "qmm_launch.h"

namespace qmm {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kShrinkThreads = 512;
constexpr int kTileRows = 16;
constexpr int kStep = 32;  // k per wavefront step of the shrink
constexpr int kMaxRank = 256;
constexpr int kNT = 4;     // 16-column tiles of a wavefront's group in the expand
constexpr int kGroupCols = kThreads / kWave * 16 * kNT;  // columns of a workgroup's group

// ---- element types: T is the storage type of A and B
struct BF16 {
    uint16_t b;
};
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(BF16 v) { return __uint_as_float((uint32_t)v.b << 16); }

// n consecutive elements at an address aligned to the whole load
template <typename T, int n>
struct alignas(sizeof(T) * n < 16 ? sizeof(T) * n : 16) Pack {
    T e[n];
};
template <typename T, int n>
__device__ __forceinline__ Pack<T, n> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, n> *>(p);
}

__device__ __forceinline__ int rank_of(const int32_t *ranks, int e, int R) {
    if (ranks == nullptr) return R;
    const int r = ranks[e];
    return r < 0 ? 0 : (r > R ? R : r);
}

// The distinct adapters of a tile, one call of f(e, match) each; match has a bit
// for every row that asks for e.  Lane l < 16 holds row l's id.  A tile that is
// shared by zsplit workgroups gives the adapter to the one that the first row
// asking for it falls to (one ballot per row of its own); otherwise the adapters
// are taken as they come, which for one adapter is one ballot.  Every wavefront of
// a workgroup sees the same ids, so f may hold barriers.
template <typename F>
__device__ __forceinline__ void for_each_adapter(int id, bool valid, int z, int zsplit, F f) {
    if (zsplit == 1) {
        uint64_t rem = __ballot(valid);
        while (rem != 0) {
            const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(rem));
            const uint64_t match = __ballot(valid && id == e);
            rem &= ~match;
            f(e, (uint32_t)match);
        }
    } else {
        for (int r = z; r < kTileRows; r += zsplit) {
            const int e = __builtin_amdgcn_readlane(id, r);
            const uint32_t match = (uint32_t)__ballot(valid && id == e);
            if (match != 0 && __builtin_ctz(match) == r) f(e, match);
        }
    }
}

// ---- v: partial sums P[s][m][r] over the k steps of split s.
// Workgroup = (tile, z, block of RT * 16 ranks, split) of eight wavefronts, which
// take pairs of the split's steps in turn and add their tiles in LDS: the partials that
// the second kernel reads again stay few.  Rows that do not match read the first
// matching row's x (same cache lines), ranks past the pool's read its last one;
// neither is used.
//
// Measured: 2048 rows, K = 8192, rank 16, two requests: 15 to 19 us for the 67 MB of
// x (3.6 to 4.4 TB/s: bound by reading x, as the second kernel of the call before it
// leaves the caches); 555 rows of seven requests, K = 4096, rank 64: 13 us, a chain
// of latencies (ids, ranks, two loads of x and A, the exchange in LDS) that a tile
// with two adapters goes through twice; 32 rows of 28 adapters, K = 8192, rank 16: 6
// us; one row: 3.7 us.
template <typename T, int RT>
__global__ __launch_bounds__(kShrinkThreads, 4) void k_lora_shrink(const T *__restrict__ A, int64_t E, int R,
                                                                const int32_t *__restrict__ ranks,
                                                                const float *__restrict__ x,
                                                                const int32_t *__restrict__ ids, int64_t M, int K,
                                                                int splits, int rank_blocks, int zsplit, int Rp,
                                                                float *__restrict__ P) {
    constexpr int W = kShrinkThreads / kWave;
    __shared__ v4f red[W][RT][kWave];
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
        // rank tiles of this block that the adapter has; with one tile the rank is not
        // waited for: whatever lies past it is not used
        const int tiles = RT == 1 ? 1 : (rank_of(ranks, e, R) - r0 + 15) >> 4;
        if (RT > 1 && tiles <= 0) return;
        const int xr = match >> row & 1 ? row : __builtin_ctz(match);
        const float *xp = x + (m0 + xr) * K + 8 * g;
        const T *ap[RT];
        v4f acc[RT];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int r = r0 + t * 16 + row;
            ap[t] = A + ((int64_t)e * R + (r < R ? r : R - 1)) * K + 8 * g;
            acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
        }
        // Loads of two steps at a time.  With one tile of ranks all of them are in flight
        // before the first products; with two, the second tile's load stands behind a
        // branch that the compiler waits in, so each step's loads come by themselves.
        constexpr int H = 2;
        for (int st = st0 + H * wave; st < st1; st += H * W) {
            const bool two = st + 1 < st1;
            Pack<float, 8> xv[H];
            Pack<T, 8> av[H][RT];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if (h == 1 && !two) break;
                xv[h] = load_pack<float, 8>(xp + (st + h) * kStep);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    if (t < tiles) av[h][t] = load_pack<T, 8>(ap[t] + (st + h) * kStep);
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if (h == 1 && !two) break;
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    if (t < tiles) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(xv[h].e[i], to_f32(av[h][t].e[i]), acc[t], 0,
                                                                          0, 0);
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < RT; ++t) red[wave][t][lane] = acc[t];
        __syncthreads();
        // element i of the tiles: float i % 4 of lane i / 4 % 64 of tile i / 256
        for (int i = threadIdx.x; i < RT * kWave * 4; i += kShrinkThreads) {
            const int t = i >> 8, l = i >> 2 & 63, q = i & 3;
            const float *p = reinterpret_cast<const float *>(&red[0][0][0]) + i;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) v += p[w * RT * kWave * 4];
            const int r = r0 + t * 16 + (l & 15), mr = 4 * (l >> 4) + q;
            if (match >> mr & 1) P[((int64_t)s * M + m0 + mr) * Rp + r] = v;
        }
        __syncthreads();
    });
}

// ---- the second product's operands.  fp32 B: C = 4 consecutive ranks per lane
// feed four v_mfma_f32_16x16x4_f32.  16-bit B: C = 8 ranks per lane feed
// v_mfma_f32_16x16x32_bf16.  v goes in as three bf16 numbers that add up to it: each
// cuts off eight bits, which is exact, and bf16 has the range of fp32, so how far
// apart the elements of a row lie does not matter (fp16 pieces under one power of
// two per row would lose the bits of an element 2^-15 of the row's largest).  A row
// whose v is small is raised by a power of two, so that small pieces do not become
// subnormal: to 2^64 for fp16 B, whose products stay below 2^89, and to 2^-64 for bf16
// B, which may be near 2^128: a sum that is finite without it stays finite (of elements
// of v below 2^-103 the last bits may be lost there).  bf16 B is used as it is.  fp16 B
// is the sum of a bf16 number of its first eight bits and one of the other three
// (subnormal ones are ordinary bf16 numbers), which is exact too.  Three products of 32
// ranks take 48 cycles, six 96; eight fp32 instructions would take 256.
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));
typedef __bf16 v8b __attribute__((ext_vector_type(8)));

// of the power of two that raises top, a row's largest |v|, to [2^to, 2^(to+1)); 0
// where it is there or above (an infinity too)
__device__ __forceinline__ int raise(float top, int to) {
    const int e = (int)(__float_as_uint(top) >> 23) - 127;  // top in [2^e, 2^(e+1)), or below 2^-126
    return e < to ? to - e : 0;
}

// the three bf16 pieces of v, the largest first
__device__ __forceinline__ void split_bf16(float v, uint16_t *p) {
    const bool finite = fabsf(v) < __builtin_inff();
    const uint32_t quiet = v != v ? 0x400000u : 0;  // cutting bits off a NaN must not leave an infinity
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = (uint16_t)((__float_as_uint(v) | quiet) >> 16);
        v = finite ? v - __uint_as_float((uint32_t)p[i] << 16) : 0.f;
    }
    if (!finite) p[1] = p[2] = 0;
}
__device__ __forceinline__ v4f mul_bf16(uint4 w, uint4 v, v4f acc) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, w), __builtin_bit_cast(v8b, v), acc, 0, 0, 0);
}

// multiply, one chunk: acc[t] += w[t] * v, the small pieces of v first
template <typename T>
struct Operand;
template <>
struct Operand<float> {
    static constexpr int C = 4, pieces = 1;
    typedef float Stored;  // v in LDS
    static __device__ __forceinline__ int exponent(float) { return 0; }
    static __device__ __forceinline__ void split(float v, Stored (&p)[1]) { p[0] = v; }
    static __device__ __forceinline__ void multiply(const uint4 (&w)[kNT], const uint4 (&v)[1], v4f (&acc)[kNT]) {
        const v4f b = __builtin_bit_cast(v4f, v[0]);
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            const v4f a = __builtin_bit_cast(v4f, w[t]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], acc[t], 0, 0, 0);
        }
    }
};
template <>
struct Operand<BF16> {
    static constexpr int C = 8, pieces = 3;
    typedef uint16_t Stored;
    static __device__ __forceinline__ int exponent(float top) { return raise(top, -64); }
    static __device__ __forceinline__ void split(float v, Stored (&p)[3]) { split_bf16(v, p); }
    static __device__ __forceinline__ void multiply(const uint4 (&w)[kNT], const uint4 (&v)[3], v4f (&acc)[kNT]) {
#pragma unroll
        for (int i = 2; i >= 0; --i)
#pragma unroll
            for (int t = 0; t < kNT; ++t) acc[t] = mul_bf16(w[t], v[i], acc[t]);
    }
};
template <>
struct Operand<_Float16> {
    // a fourth piece: the first with 0 for what is not finite, for the low part of B.  An
    // infinite v times the high part is the result; times the low part, which is often
    // 0 and may have the other sign, it would make a NaN of it.
    static constexpr int C = 8, pieces = 4;
    typedef uint16_t Stored;
    static __device__ __forceinline__ int exponent(float top) { return raise(top, 64); }
    static __device__ __forceinline__ void split(float v, Stored (&p)[4]) {
        split_bf16(v, p);
        p[3] = fabsf(v) < __builtin_inff() ? p[0] : 0;
    }
    static __device__ __forceinline__ void halves(uint32_t two, uint32_t &high, uint32_t &low) {
        const v2h h = __builtin_bit_cast(v2h, two);
        const float a = (float)h[0], b = (float)h[1];
        high = __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2b));
        const float ra = a - __uint_as_float(high << 16), rb = b - __uint_as_float(high & 0xffff0000u);
        low = __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{ra, rb}, v2b));
    }
    static __device__ __forceinline__ void multiply(const uint4 (&w)[kNT], const uint4 (&v)[4], v4f (&acc)[kNT]) {
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            uint4 high, low;
            halves(w[t].x, high.x, low.x);
            halves(w[t].y, high.y, low.y);
            halves(w[t].z, high.z, low.z);
            halves(w[t].w, high.w, low.w);
#pragma unroll
            for (int i = 2; i >= 0; --i) {
                acc[t] = mul_bf16(low, i == 0 ? v[3] : v[i], acc[t]);
                acc[t] = mul_bf16(high, v[i], acc[t]);
            }
        }
    }
};

// elements of a row of v in LDS: whole chunks of 4 * C ranks, and 16 bytes more so
// that the rows start on different banks
template <typename T>
__host__ __device__ constexpr int v_row(int Rp) {
    return (Rp + 4 * Operand<T>::C - 1) / (4 * Operand<T>::C) * (4 * Operand<T>::C) +
           16 / (int)sizeof(typename Operand<T>::Stored);
}

// The sixteen lanes of a row add up its Rp ranks' partials in groups of 4, 8 or 16: log2
// of a group's lanes.
__host__ __device__ constexpr int part_lanes(int Rp) { return Rp <= 16 ? 2 : (Rp <= 32 ? 3 : 4); }

// ---- out = base + v B^T.  Workgroup = (tile, z, strip of columns).  The tile's v
// (partials added in order, scaled, each row with its own adapter's rank) goes to
// LDS once.  Per group of 256 columns each wavefront multiplies four times 16
// columns of B, adapter by adapter: B's rows are the matrix instruction's rows, so
// a lane ends with four consecutive columns of one output row, and the rows that
// match go to a tile in LDS.  From there base and out are read and written by
// whole rows, 1 KiB per wavefront and instruction.  The first group's base is asked for
// before the partials (by tiles that are not shared), its B behind them: it arrives
// while v is scaled and cut.  VEC: rows of base and out are 16-byte
// aligned and N is a multiple of 4 (16-byte accesses); GR: R is a multiple of it (B
// in loads of GR elements: C, C / 2, C / 4 or 1); H: 64 * H ranks at most (GR < C is
// built with H = 4 alone: the loops over h end at the rank all the same).
//
// Measured (base and out not in a cache): 2048 rows, N = 28672, rank 16, fp16 B: 84 us
// of the 79 that adding two matrices of this size takes, 5.6 TB/s; 555 rows, rank 64, bf16: 37 us, of which the partials take 5 (32 KB of
// them per workgroup, out of the L2) and B 4; 127 MB of base and out alone would take 21;
// 32 rows of 28 adapters, N = 8192: 7.9 us; one row, N = 4096, fp16: 5.1 us, a chain of
// ids, partials, B and the exchange of the tile.
//
// Shared (zsplit > 1) has the registers of three workgroups per CU, not four: fp16 B
// and ranks that are no multiple of C spill otherwise (64 rows of 16 adapters, rank
// 64, N = 28672, fp16: 35.0 -> 31.8 us; 100 rows at rank 12: 36.8 -> 32.2 us).  So do
// 16-bit B of odd ranks, read by single elements: fp16 (2048 rows of 28672 at rank 33:
// 228 -> 220 us), and bf16 where rows are not 16-byte aligned (of 28671: 261 -> 236 us;
// aligned ones fit, 212 us against 217).
enum class Tiles { Own, Shared, Long };  // Shared: zsplit > 1; Long: base and out go past the caches
template <typename T, bool VEC, int GR, Tiles MODE>
constexpr int expand_workgroups =
    MODE == Tiles::Shared || (GR == 1 && (__is_same(T, _Float16) || (__is_same(T, BF16) && !VEC))) ? 3 : 4;
template <typename T, bool VEC, int GR, int H, Tiles MODE>
__global__ __launch_bounds__(kThreads, (expand_workgroups<T, VEC, GR, MODE>)) void k_lora_expand(const T *__restrict__ B, int64_t E, int R,
                                                          const float *__restrict__ scales,
                                                          const int32_t *__restrict__ ranks,
                                                          const int32_t *__restrict__ ids, int64_t M,
                                                          const float *__restrict__ P, int splits, int Rp,
                                                          const float *base, int64_t ld_base, float *out,
                                                          int64_t ld_out, int64_t N, int strips, int groups,
                                                          int zsplit) {
    typedef Operand<T> Op;
    typedef typename Op::Stored Stored;
    constexpr bool SHARED = MODE == Tiles::Shared;
    constexpr int C = Op::C;
    constexpr int kTileLd = kGroupCols + 4;
    constexpr int kRows = kTileRows / (kThreads / kWave);  // output rows of a wavefront
    __shared__ __align__(16) float tile[kTileRows * kTileLd];
    __shared__ int exponents[kTileRows];
    extern __shared__ __align__(16) uint8_t v_lds[];  // Stored [pieces][kTileRows][vld]
    Stored *vs = reinterpret_cast<Stored *>(v_lds);
    const int vld = v_row<T>(Rp);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane & 15, g = lane >> 4;
    uint32_t b = blockIdx.x;
    const int64_t strip0 = (int64_t)(b % strips) * groups * kGroupCols;
    b /= strips;
    const int z = SHARED ? (int)(b % (uint32_t)zsplit) : 0;
    const int64_t m0 = (int64_t)(SHARED ? b / zsplit : b) * kTileRows;
    const int tile_rows = M - m0 < kTileRows ? (int)(M - m0) : kTileRows;
    // Loads below take the nearest valid address where theirs is past an end, and
    // what they bring there is not used: no branch stands between them, so a wait
    // for one does not become a wait for all.
    // lane l holds what row l % 16 asks for
    int id = ids[m0 + (row < tile_rows ? row : tile_rows - 1)];

    // this wavefront's rows of base: four consecutive columns per lane, or columns
    // lane, lane + 64, ...
    v4f o[kRows];
    auto column = [&](int64_t n0, int q) { return n0 + (VEC ? 4 * lane + q : lane + 64 * q); };
    auto load_base = [&](int64_t n0, uint32_t rows) {
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int mr = wave * kRows + i;
            if (SHARED && !(rows >> mr & 1)) continue;  // other workgroups' rows
            const float *p = base + (m0 + (mr < tile_rows ? mr : tile_rows - 1)) * ld_base;
            if (VEC) {
                const int64_t n = column(n0, 0);
                const v4f *at = reinterpret_cast<const v4f *>(p + (n < N ? n : N - 4));
                o[i] = MODE == Tiles::Long ? __builtin_nontemporal_load(at) : *at;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t n = column(n0, q);
                    o[i][q] = p[n < N ? n : N - 1];
                }
            }
        }
    };
    // a tile that is not shared is read before it is known who wants what
    if (!SHARED) load_base(strip0, ~0u);

    id = row < tile_rows ? id : -1;
    const bool valid = id >= 0 && id < E;
    // the rows this workgroup writes: those of its adapters, and for z = 0 the ones
    // without (in place these stay as they are)
    uint32_t here = 0;
    const int of = SHARED ? zsplit : 1;
    for_each_adapter(id, valid && lane < kTileRows, z, of, [&](int, uint32_t match) { here |= match; });
    const uint32_t adapters = here;
    if (z == 0)
        here |= (uint32_t)__ballot(lane < tile_rows && !valid && !(id == -1 && base == out));
    if (here == 0) return;
    const int own = valid ? id : 0;
    int rank = R;
    float scale = 1.0f;
    if (ranks != nullptr) rank = ranks[own];
    if (scales != nullptr) scale = scales[own];

    // C ranks from r on (16 bytes) of this lane's rows of B in the wavefront's columns
    uint4 w[kNT];
    auto load_b = [&](int e, int64_t n0, int r) {
        const T *Be = B + ((int64_t)e * N + n0) * R;
        const int cols = N - n0 < kGroupCols ? (int)(N - n0) : kGroupCols;
#pragma unroll
        for (int t = 0; t < kNT; ++t) {
            const int nb = (wave * kNT + t) * 16 + row;
            const T *p = Be + (uint32_t)((nb < cols ? nb : cols - 1) * R);
            if constexpr (GR == C) {
                w[t] = ld16(p + (r < R ? r : 0));
            } else if constexpr (GR == C / 2) {
                const uint2 a = *reinterpret_cast<const uint2 *>(p + (r < R ? r : 0));
                const uint2 b = *reinterpret_cast<const uint2 *>(p + (r + GR < R ? r + GR : 0));
                w[t] = make_uint4(a.x, a.y, b.x, b.y);
            } else if constexpr (GR == C / 4) {
                uint32_t q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = r + i * GR < R ? r + i * GR : 0;
                    q[i] = *reinterpret_cast<const uint32_t *>(p + at);
                }
                w[t] = make_uint4(q[0], q[1], q[2], q[3]);
            } else {
                Pack<T, C> q;
#pragma unroll
                for (int i = 0; i < C; ++i) q.e[i] = p[r + i < R ? r + i : 0];
                w[t] = __builtin_bit_cast(uint4, q);
            }
        }
    };

    // v's partials: sixteen lanes per row, four consecutive ranks each and 64 at a
    // time; with 16 or 32 ranks in all, four or two groups of lanes take every fourth
    // or second part (the workspace has room for whole groups of them; Long has few
    // parts and does without, 96.2 against 97.7 us at 2048 x 28672 with 4 of them, though
    // 42.8 against 41.6 us at 700 x 28672 with 12).  A row without
    // an adapter has none, what is read there and past the last part is not used
    const int vrow = wave * kRows + g;  // kRows is 4: the wavefront's rows by 16 lanes each
    v4f v[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        const int shift = h > 0 || MODE == Tiles::Long ? 4 : part_lanes(Rp), step = 16 >> shift;
        const int r = 64 * h + 4 * (row & ((1 << shift) - 1)), mine = row >> shift;
        const float *p = P + (mine * M + m0 + (vrow < tile_rows ? vrow : tile_rows - 1)) * Rp + (r < Rp ? r : 0);
        v[h] = v4f{0.f, 0.f, 0.f, 0.f};
        if (64 * h >= Rp) break;
        for (int s = 0; s < splits; s += 8 * step) {
            v4f part[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                part[i] = *reinterpret_cast<const v4f *>(p + (int64_t)(s + i * step < splits ? s + i * step : s) * M * Rp);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[h] += s + i * step + mine < splits ? part[i] : v4f{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {  // groups 8 lanes apart, then 4: every lane adds the same pairs
            if (step > 1) v[h][q] += dpp_f32<0x128>(v[h][q]);
            if (step > 2) v[h][q] += dpp_f32<0x124>(v[h][q]);
        }
    }
    // the first group's B, and base of a shared tile, arrive while v is scaled and cut
    const int first = adapters != 0 ? __builtin_ctz(adapters) : 0;  // a row of the first adapter
    load_b(__builtin_amdgcn_readlane(own, first), strip0, C * g);
    if (SHARED) load_base(strip0, here);
    rank = !valid || rank < 0 ? 0 : (rank > R ? R : rank);
    {
        int rk = __shfl(rank, vrow);  // every lane takes part: the source lane has to be active
        const float sc = __shfl(scale, vrow);
        rk = adapters >> vrow & 1 ? rk : 0;
        float top = 0.f;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[h][q] = 64 * h + 4 * row + q < rk ? v[h][q] * sc : 0.f;
                top = fmaxf(top, fabsf(v[h][q]));
            }
        top = fmaxf(top, dpp_f32<0xB1>(top));  // over the row's sixteen lanes
        top = fmaxf(top, dpp_f32<0x4E>(top));
        top = fmaxf(top, dpp_f32<0x141>(top));
        top = fmaxf(top, dpp_f32<0x140>(top));
        const int ex = Op::exponent(top);
        if (row == 0) exponents[vrow] = -ex;
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int r = 64 * h + 4 * row;
            if (r >= vld) continue;  // past what the chunks of 4 * C ranks read
            Stored p4[4][Op::pieces];
#pragma unroll
            for (int q = 0; q < 4; ++q) Op::split(Op::pieces > 1 ? ldexpf(v[h][q], ex) : v[h][q], p4[q]);
#pragma unroll
            for (int i = 0; i < Op::pieces; ++i) {
                const Pack<Stored, 4> four{{p4[0][i], p4[1][i], p4[2][i], p4[3][i]}};
                *reinterpret_cast<Pack<Stored, 4> *>(vs + (i * kTileRows + vrow) * vld + r) = four;
            }
        }
    }
    __syncthreads();

    for (int j = 0; j < groups; ++j) {
        const int64_t n0 = strip0 + (int64_t)j * kGroupCols;
        for_each_adapter(id, valid && lane < kTileRows, z, of, [&](int e, uint32_t match) {
            const int er = __builtin_amdgcn_readlane(rank, __builtin_ctz(match));
            v4f acc[kNT];
#pragma unroll
            for (int t = 0; t < kNT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};
            for (int c = 0; c < er; c += 4 * C) {
                const int r = c + C * g;
                if (j > 0 || c > 0 || !(match >> first & 1)) load_b(e, n0, r);
                if (c + 4 * C > er) {  // what B holds behind the rank is not used
                    uint32_t keep[4];
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        const int left = er - r - d * (C / 4);
                        keep[d] = left >= C / 4 ? ~0u : (left == 1 ? 0xffffu : 0u);
                    }
#pragma unroll
                    for (int t = 0; t < kNT; ++t)
                        w[t] = make_uint4(w[t].x & keep[0], w[t].y & keep[1], w[t].z & keep[2], w[t].w & keep[3]);
                }
                uint4 vp[Op::pieces];
#pragma unroll
                for (int i = 0; i < Op::pieces; ++i) vp[i] = ld16(vs + (i * kTileRows + row) * vld + r);
                Op::multiply(w, vp, acc);
            }
            if (match >> row & 1) {
                const int ex = exponents[row];
#pragma unroll
                for (int t = 0; t < kNT; ++t) {
                    if (Op::pieces > 1)
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[t][q] = ldexpf(acc[t][q], ex);
                    *reinterpret_cast<v4f *>(&tile[row * kTileLd + (wave * kNT + t) * 16 + 4 * g]) = acc[t];
                }
            }
        });
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int mr = wave * kRows + i;
            if (!(here >> mr & 1)) continue;
            const int e = __builtin_amdgcn_readlane(id, mr);
            const float *d = &tile[mr * kTileLd];
            float *p = out + (m0 + mr) * ld_out;
            if (e >= 0 && e < E) {
                if (VEC) {
                    o[i] += *reinterpret_cast<const v4f *>(d + 4 * lane);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q) o[i][q] += d[lane + 64 * q];
                }
            } else if (e != -1) {
                const float nan = __builtin_nanf("");
                o[i] = v4f{nan, nan, nan, nan};
            }
            if (VEC) {
                v4f *to = reinterpret_cast<v4f *>(p + column(n0, 0));
                if (column(n0, 0) < N && MODE == Tiles::Long) __builtin_nontemporal_store(o[i], to);
                else if (column(n0, 0) < N) *to = o[i];
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (column(n0, q) < N) p[column(n0, q)] = o[i][q];
            }
        }
        if (j + 1 == groups || n0 + kGroupCols >= N) break;
        load_base(n0 + kGroupCols, here);
        __syncthreads();
    }
}

// ---- launch shapes (host only; they need no device)
constexpr int kMaxSplits = 32;

struct Shape {
    int rt, rank_blocks, Rp, zsplit, splits;
    int64_t tiles;
};
Shape shape(int64_t M, int64_t R, int64_t K, int64_t E) {
    Shape h;
    // a second tile of ranks uses the same x; four in one workgroup are slower than two
    // workgroups of two (512 rows, K = 14336, rank 64: 79 us for both kernels, 67 so)
    h.rt = R <= 16 ? 1 : 2;
    h.rank_blocks = (int)((R + 16 * h.rt - 1) / (16 * h.rt));
    h.Rp = h.rank_blocks * h.rt * 16;
    h.tiles = (M + kTileRows - 1) / kTileRows;
    // Adapters of a tile side by side pay where a tile has many and there are few
    // tiles; workgroups without an adapter cost what it takes to start them, and how
    // many adapters a tile has is not known here.  Both kernels, K = 4096, N = 4096,
    // rank 16, parts 16 / 4 / 1 of a tile: 48 rows of 16 requests 11.5 / 12.4 / 18.6
    // us, of one 12.3 / 10.9 / 10.9; 100 rows of 64 requests - / 16.1 / 29.5, of one
    // - / 10.8 / 11.0; 256 rows of 64 - / 19.0 / 19.2, of one - / 14.3 / 11.1
    h.zsplit = M <= 32 ? 16 : (M <= 128 ? 4 : 1);
    if (h.zsplit > E) h.zsplit = (int)E;
    if (h.zsplit > M) h.zsplit = (int)M;
    // two workgroups of eight wavefronts per CU, four where some of them may find no
    // adapter or no rank of theirs (256 rows, K = 14336, rank 128: 65 us with four, 100
    // with two; 700 rows at rank 32: 32 with two, 36 with four), and two steps for
    // each wavefront at least
    const int64_t groups = h.tiles * h.zsplit * h.rank_blocks;
    const int64_t most = (K / kStep + 2 * (kShrinkThreads / kWave) - 1) / (2 * (kShrinkThreads / kWave));
    const int64_t wanted = h.zsplit > 1 || h.rank_blocks > 1 ? 1024 : 512;
    int64_t s = (wanted + groups - 1) / groups;
    s = s > kMaxSplits ? kMaxSplits : s;
    h.splits = (int)(s > most ? most : s);
    return h;
}
// Column groups per workgroup of the second kernel: two where workgroups are plenty
// all the same, so that each adds up the partials once for both (both kernels, K =
// 4096, rank 16: 1024 rows of 28672 columns 53.9 -> 49.3 us, 800 rows 43.5 -> 41.5 us;
// three: 45.5 us; from 1024 groups on 40 rows of 28672 would take 14.2 instead of 12.3
// us)
struct Strips {
    int64_t strips;
    int groups;
};
Strips strips_of(int64_t N, const Shape &h) {
    const int64_t all = (N + kGroupCols - 1) / kGroupCols;
    const int groups = all * h.tiles * h.zsplit >= 2048 ? 2 : 1;
    return Strips{(all + groups - 1) / groups, groups};
}

template <typename T, int RT>
hipError_t shrink(const LoraArgs &a, const Shape &h, hipStream_t s) {
    const int64_t grid = h.tiles * h.zsplit * h.rank_blocks * h.splits;
    hipLaunchKernelGGL((k_lora_shrink<T, RT>), dim3((unsigned)grid), dim3(kShrinkThreads), 0, s,
                       static_cast<const T *>(a.A), a.E, (int)a.R, a.ranks, a.x, a.ids, a.M, (int)a.K, h.splits,
                       h.rank_blocks, h.zsplit, h.Rp, a.ws);
    return hipGetLastError();
}

template <typename T, bool VEC, int GR, int H>
hipError_t expand(const LoraArgs &a, const Shape &h, hipStream_t s) {
    const Strips st = strips_of(a.N, h);
    const size_t lds = sizeof(typename Operand<T>::Stored) * Operand<T>::pieces * kTileRows * v_row<T>(h.Rp);
    // 32 MiB of out are more than the L2 caches hold: it goes past them, and base with it
    // (2048 rows of 28672: 105 -> 101 us for both kernels, 555 rows at rank 64: 55 -> 50
    // us, inputs in turn).  In place on what a kernel before it wrote and read by a
    // quantization after it, plain accesses are 1 to 2% faster up to 128 MiB, which the
    // 256 MB cache behind the L2 holds (1100 rows of 8192: 45.2 us for the three kernels
    // against 45.7), past the caches 2 to 5% from 224 MiB on (8192 rows: 263 against 277).
    const auto kernel = h.zsplit > 1 ? k_lora_expand<T, VEC, GR, H, Tiles::Shared>
                        : VEC && a.M * a.N >= (int64_t(32) << 20) / 4
                            ? k_lora_expand<T, VEC, GR, H, VEC ? Tiles::Long : Tiles::Own>
                            : k_lora_expand<T, VEC, GR, H, Tiles::Own>;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(st.strips * h.zsplit * h.tiles)), dim3(kThreads), lds, s,
                       static_cast<const T *>(a.B), a.E, (int)a.R, a.scales, a.ranks, a.ids, a.M, a.ws, h.splits, h.Rp,
                       a.base, a.ld_base, a.out, a.ld_out, a.N, (int)st.strips, st.groups, h.zsplit);
    return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t expand_for(const LoraArgs &a, const Shape &h, hipStream_t s) {
    constexpr int H = kMaxRank / 64, C = Operand<T>::C;
    if (a.R % C == 0) return h.Rp <= 64 ? expand<T, VEC, C, 1>(a, h, s) : expand<T, VEC, C, H>(a, h, s);
    // wider pieces of a lane's 16 bytes of B than single elements (2048 rows, N = 28672:
    // rank 60 in fp16 277 us by elements, 143 us by 8 bytes)
    if (a.R % (C / 2) == 0) return expand<T, VEC, C / 2, H>(a, h, s);
    if (a.R % (C / 4) == 0) return expand<T, VEC, C / 4, H>(a, h, s);
    return expand<T, VEC, 1, H>(a, h, s);
}

template <typename T>
hipError_t both(const LoraArgs &a, hipStream_t s) {
    const Shape h = shape(a.M, a.R, a.K, a.E);
    const hipError_t e = h.rt == 1 ? shrink<T, 1>(a, h, s) : shrink<T, 2>(a, h, s);
    if (e != hipSuccess) return e;
    const bool vec = a.ld_base % 4 == 0 && a.ld_out % 4 == 0 && a.N % 4 == 0;
    return vec ? expand_for<T, true>(a, h, s) : expand_for<T, false>(a, h, s);
}

}  // namespace

int64_t lora_workspace_bytes(int64_t M, int64_t R, int64_t K, int64_t E) {
    const Shape h = shape(M, R, K, E);
    const int g = 16 >> part_lanes(h.Rp);
    return (int64_t)sizeof(float) * ((h.splits + g - 1) / g * g) * M * h.Rp;
}

int64_t lora_max_rank() { return kMaxRank; }

void lora_shape(int64_t M, int64_t R, int64_t K, int64_t E, int *splits, int *shared) {
    const Shape h = shape(M, R, K, E);
    *splits = h.splits;
    *shared = h.zsplit;
}

bool lora_grid_ok(int64_t M, int64_t N, int64_t R, int64_t K, int64_t E) {
    const Shape h = shape(M, R, K, E);
    const int64_t threads = int64_t(1) << 32;  // of one launch: they are counted in 32 bits
    return h.tiles * h.zsplit * h.rank_blocks * h.splits * kShrinkThreads < threads &&
           strips_of(N, h).strips * h.zsplit * h.tiles * kThreads < threads;
}

hipError_t launch_lora_add(int type, const LoraArgs &a, hipStream_t s) {
    switch (type) {
        case 0: return both<float>(a, s);
        case 1: return both<_Float16>(a, s);
        default: return both<BF16>(a, s);
    }
}

}  // namespace qmm
