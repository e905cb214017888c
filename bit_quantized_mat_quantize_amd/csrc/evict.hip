// evict.hip -- a cache within its budget (gfx950): per sequence and head the newest
// entries and, of the others, those of the most accumulated weight, ties to the
// lower index; what stays moves together in its order.
//
// k_evict_select, one workgroup per (sequence, head): the weights' bits, mapped to
// unsigned keys of the same order, by radix select in digits of 11, 11 and 10 bits (a
// histogram in LDS each: integer counts, so their order does not matter), which gives the
// key of the last entry that stays and how many of its equals do; then the places
// of what stays by ballots and a sum over wavefronts, in the entries' order.  The keys
// stay in registers up to 16384 entries.
//
// 128 times 9000 keys: 13.3 us.  Read anew in each pass, 8 x 8 times 16000 keys took the
// whole call from 67 to 83 us.
//
// k_evict_move: entries in ascending order.  Into other pages every chunk has a workgroup
// of its own.  Within the same pages one workgroup per (sequence, head, keys or
// values) goes through them, all of a chunk in registers before any of it is
// stored: an entry only ever moves down, so chunks yet to be read lie above everything
// stored before.  Bound by HBM (16 x 4096 entries of 8 heads of 128 into other pages: 42.3
// us, 3.6 TB/s read and written; entries that stay lie apart, and cache lines are read
// for the 64 bytes of one), within the same pages of few sequences and heads by the chain of one
// workgroup's chunks: both kernels in the sequences' own pages and into others, 8 heads of 128: 16 x 9000 -> 4096
// entries 54.7 and 47.4 us, 8 x 16000 -> 12000 114 and 65, 4 x 1100 -> 1024 18.7 and 13.5, one of 131072 -> 65536 684
// and 198.
#include "kv_device.h"

namespace qmm {
namespace {

constexpr int kSelect = 1024, kWaves = kSelect / 64, kBins = 2048;
constexpr int kMove = 256;

// larger keys for larger weights, -0 as 0, NaN above all
__device__ __forceinline__ uint32_t order_key(float m) {
    if (m != m) return 0xffffffffu;
    const uint32_t u = __float_as_uint(m + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// KEYS: entries per thread that stay in registers (0: none do, they are read anew)
template <int KEYS>
__global__ __launch_bounds__(kSelect) void k_evict_select(EvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t sums[2][KEYS > 1 ? KEYS : 1][kWaves];
    __shared__ uint32_t found[2];  // the digit, and what is left to take within it
    const int h = blockIdx.x % a.c.heads, b = blockIdx.x / a.c.heads, tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int most = a.c.width << a.c.page_log2, given = a.c.lens[b];
    const int L = given < 0 ? 0 : (given > most ? most : given), n = L < a.budget ? L : a.budget;
    const float *mass = a.mass + ((int64_t)b * a.c.heads + h) * a.ld_mass;
    float *mass_out = a.mass_out + ((int64_t)b * a.c.heads + h) * a.ld_out;
    int32_t *ids = a.ids + ((int64_t)b * a.c.heads + h) * a.budget;
    if (h == 0 && tid == 0) a.lens_out[b] = n;
    for (int i = n + tid; i < a.budget; i += kSelect) ids[i] = -1;
    for (int64_t i = n + tid; i < a.ld_out; i += kSelect) mass_out[i] = 0.0f;
    if (L <= a.budget) {
        for (int i = tid; i < L; i += kSelect) {
            ids[i] = i;
            mass_out[i] = mass[i];
        }
        return;
    }
    const int old = L - a.recent, need = a.budget - a.recent;  // recent <= budget < L
    float m[KEYS > 0 ? KEYS : 1];
    if constexpr (KEYS > 0) {
#pragma unroll
        for (int j = 0; j < KEYS; ++j) m[j] = j * kSelect + tid < old ? mass[j * kSelect + tid] : 0.0f;
    }
    for (int i = tid; i < a.recent; i += kSelect) {
        ids[need + i] = old + i;
        mass_out[need + i] = mass[old + i];
    }
    if (need == 0) return;
    // f(position, weight) for this thread's entries among the old ones
    auto each = [&](auto f) {
        if constexpr (KEYS > 0) {
#pragma unroll
            for (int j = 0; j < KEYS; ++j)
                if (j * kSelect + tid < old) f(j * kSelect + tid, m[j]);
        } else
            for (int i = tid; i < old; i += kSelect) f(i, mass[i]);
    };
    uint32_t prefix = 0, left = need;  // the key's digits found so far; entries to take among those that share them
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        reinterpret_cast<uint2 *>(hist)[tid] = make_uint2(0, 0);
        __syncthreads();
        each([&](int, float w) {
            const uint32_t key = order_key(w);
            if (pass == 0 || (key >> (shift + bits)) == prefix) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
        });
        __syncthreads();
        // from the largest digit down: thread i has two bins
        const uint2 c = reinterpret_cast<const uint2 *>(hist)[kSelect - 1 - tid];  // .y is the larger one
        uint32_t upto = c.x + c.y;
        for (int o = 1; o < 64; o <<= 1) {
            const uint32_t up = __shfl_up(upto, o, 64);
            if (lane >= o) upto += up;
        }
        if (lane == 63) sums[0][0][wave] = upto;
        __syncthreads();
        uint32_t before = upto - c.x - c.y;
        for (int w = 0; w < wave; ++w) before += sums[0][0][w];
        const int bin = kBins - 1 - 2 * tid;
        if (before < left && before + c.y >= left) {
            found[0] = bin;
            found[1] = left - before;
        } else if (before + c.y < left && before + c.y + c.x >= left) {
            found[0] = bin - 1;
            found[1] = left - before - c.y;
        }
        __syncthreads();
        prefix = (prefix << bits) | found[0];
        left = found[1];
    }
    // entries above the key stay, and the first `left` of those that equal it
    const uint64_t below = (uint64_t(1) << lane) - 1;
    if constexpr (KEYS > 0) {
#pragma unroll
        for (int j = 0; j < KEYS; ++j) {
            const uint32_t key = order_key(m[j]);
            const bool in = j * kSelect + tid < old;
            const uint32_t above = __popcll(__ballot(in && key > prefix)), equal = __popcll(__ballot(in && key == prefix));
            if (lane == 0) {
                sums[0][j][wave] = above;
                sums[1][j][wave] = equal;
            }
        }
        __syncthreads();
        // of all runs of 64 entries before each: the first wavefront adds them up
        if (wave == 0) {
            uint32_t above = 0, equal = 0;  // before this lane's runs
            constexpr int RUNS = KEYS * kWaves, PER = (RUNS + 63) / 64;
            uint32_t va[PER], ve[PER], ta = 0, te = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = lane * PER + i;
                va[i] = r < RUNS ? (&sums[0][0][0])[r] : 0;
                ve[i] = r < RUNS ? (&sums[1][0][0])[r] : 0;
                ta += va[i];
                te += ve[i];
            }
            above = ta, equal = te;
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t ua = __shfl_up(above, o, 64), ue = __shfl_up(equal, o, 64);
                if (lane >= o) above += ua, equal += ue;
            }
            above -= ta;
            equal -= te;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int r = lane * PER + i;
                if (r < RUNS) {
                    (&sums[0][0][0])[r] = above;
                    (&sums[1][0][0])[r] = equal;
                }
                above += va[i];
                equal += ve[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < KEYS; ++j) {
            const uint32_t key = order_key(m[j]), equals = sums[1][j][wave];
            const bool in = j * kSelect + tid < old;
            const uint64_t eq = __ballot(in && key == prefix);
            const bool stays = in && (key > prefix || (key == prefix && equals + __popcll(eq & below) < left));
            const uint64_t all = __ballot(stays);
            if (stays) {
                const uint32_t at = sums[0][j][wave] + (equals < left ? equals : left) + __popcll(all & below);
                ids[at] = j * kSelect + tid;
                mass_out[at] = m[j];
            }
        }
    } else {
        const int per = ((old + kSelect - 1) / kSelect) * 64;  // positions of a wavefront
        const int p0 = wave * per, p1 = p0 + per < old ? p0 + per : old;
        uint32_t above = 0, equal = 0;
        for (int i = p0; i < p1; i += 64) {
            const bool in = i + lane < p1;
            const uint32_t key = in ? order_key(mass[i + lane]) : 0;
            above += __popcll(__ballot(in && key > prefix));
            equal += __popcll(__ballot(in && key == prefix));
        }
        if (lane == 0) {
            sums[0][0][wave] = above;
            sums[1][0][wave] = equal;
        }
        __syncthreads();
        uint32_t taken = 0, equals = 0;
        for (int w = 0; w < wave; ++w) {
            taken += sums[0][0][w];
            equals += sums[1][0][w];
        }
        taken += equals < left ? equals : left;
        for (int i = p0; i < p1; i += 64) {
            const bool in = i + lane < p1;
            const float w = in ? mass[i + lane] : 0.0f;
            const uint32_t key = order_key(w);
            const uint64_t eq = __ballot(in && key == prefix);
            const bool stays = in && (key > prefix || (key == prefix && equals + __popcll(eq & below) < left));
            const uint64_t all = __ballot(stays);
            if (stays) {
                const uint32_t at = taken + __popcll(all & below);
                ids[at] = i + lane;
                mass_out[at] = w;
            }
            taken += __popcll(all);
            equals += __popcll(eq);
        }
    }
}

// a value that another thread's store may replace: read for good before the barrier
__device__ __forceinline__ void arrived(uint4 &v, uint32_t &s) {
    asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w), "+v"(s));
}

// entries at a time: one 16-byte piece of codes and one scale per thread, values in fours
__host__ __device__ constexpr int move_chunk(int threads, int D) { return threads / (D / 32) & ~3; }
// chunks of a sequence and head, of kMove threads each
int64_t move_parts(int64_t D, int64_t capacity, int64_t budget) {
    const int chunk = move_chunk(kMove, (int)D);
    return ((capacity < budget ? capacity : budget) + chunk - 1) / chunk;
}

// CHAIN: one workgroup goes through all chunks (the same pages), the places of the one after
// the next, the codes of the next and the stores of this one at a time; else it has one.
template <bool CHAIN, int THREADS>
__global__ __launch_bounds__(THREADS) void k_evict_move(EvictArgs a, int parts) {
    __shared__ int2 from[CHAIN ? 3 : 1][THREADS / 2];  // page (-1: none) and entry that a chunk's entries come from
    const int x = CHAIN ? blockIdx.x : blockIdx.x / parts;
    const int part = x & 1, h = (x >> 1) % a.c.heads, b = (x >> 1) / a.c.heads;
    const int D = a.c.D, nb = D / 32, lg = a.c.page_log2, mask = (1 << lg) - 1;
    const int32_t *ids = a.ids + ((int64_t)b * a.c.heads + h) * a.budget;
    const int32_t *table = a.c.table + (int64_t)b * a.c.width, *to = a.to + (int64_t)b * a.to_width;
    const int most = a.c.width << lg, given = a.c.lens[b];
    const int L = given < 0 ? 0 : (given > most ? most : given), n = L < a.budget ? L : a.budget;
    const int chunk = move_chunk(THREADS, D);
    const int tid = threadIdx.x, words = D / 8;
    const bool active = tid < chunk * nb;
    // keys: piece p of entry j; values: word w of the entries 4g .. 4g + 3; scales: block s of entry i
    const int j = active ? tid / nb : 0, p = tid - j * nb, g = active ? tid / words : 0, w = tid - g * words;
    const int s = active ? tid / chunk : 0, i = tid - s * chunk;
    auto places = [&](int c0, int slot) {
        if (tid >= chunk) return;
        int2 f = make_int2(-1, 0);
        if (c0 + tid < n) {
            const int id = ids[c0 + tid], page = table[id >> lg];
            f = make_int2(page >= 0 && page < a.c.pages ? page : -1, id & mask);
        }
        from[slot][tid] = f;
    };
    auto read = [&](int slot, uint4 &v, uint32_t &scale) {
        v = make_uint4(0, 0, 0, 0);
        scale = 0x7e00u;  // an entry whose page is not there is NaN
        if (!active) return;
        if (part == 0) {
            const int2 f = from[slot][j];
            if (f.x >= 0) v = ld16(kv_chunk(a.c, f.x, 0, h) + f.y * (D / 2) + p * 16);
        } else {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int2 f = from[slot][4 * g + e];
                u[e] = f.x >= 0 ? reinterpret_cast<const uint32_t *>(kv_chunk(a.c, f.x, 1, h))[kv_value_word(D, f.y, w)] : 0;
            }
            v = make_uint4(u[0], u[1], u[2], u[3]);
        }
        const int2 f = from[slot][i];
        if (f.x >= 0) scale = reinterpret_cast<const uint16_t *>(kv_chunk(a.c, f.x, part, h))[kv_scale_at(a.c, f.y, s)];
    };
    auto target = [&](int at) -> uint8_t * {
        if (at >= n) return nullptr;
        const int page = to[at >> lg];
        return page >= 0 && page < a.c.pages ? kv_chunk(a.c, page, part, h) : nullptr;
    };
    auto write = [&](int c0, const uint4 &v, uint32_t scale) {
        if (!active) return;
        if (part == 0) {
            const int at = c0 + j;
            if (uint8_t *q = target(at)) *reinterpret_cast<uint4 *>(q + (at & mask) * (D / 2) + p * 16) = v;
        } else {
            const int at = c0 + 4 * g;
            if (uint8_t *q = target(at)) {
                uint32_t *o = reinterpret_cast<uint32_t *>(q) + kv_value_word(D, at & mask, w);
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                if (at + 4 <= n) *reinterpret_cast<uint4 *>(o) = v;
                else
#pragma unroll
                    for (int e = 0; e < 3; ++e)
                        if (at + e < n) o[e] = u[e];
            }
        }
        const int at = c0 + i;
        if (uint8_t *q = target(at)) reinterpret_cast<uint16_t *>(q)[kv_scale_at(a.c, at & mask, s)] = (uint16_t)scale;
    };
    if constexpr (!CHAIN) {
        const int c0 = (blockIdx.x - x * parts) * chunk;
        if (c0 >= n) return;
        uint4 v;
        uint32_t scale;
        places(c0, 0);
        __syncthreads();
        read(0, v, scale);
        write(c0, v, scale);
    } else {
        uint4 v, next;
        uint32_t scale, next_scale;
        places(0, 0);
        places(chunk, 1);
        __syncthreads();
        read(0, v, scale);
        for (int c0 = 0, k = 0; c0 < n; c0 += chunk, ++k) {
            read((k + 1) % 3, next, next_scale);
            places(c0 + 2 * chunk, (k + 2) % 3);
            arrived(v, scale);
            __syncthreads();
            write(c0, v, scale);
            v = next;
            scale = next_scale;
        }
    }
}

}  // namespace

int64_t evict_workgroups(int64_t B, int64_t heads, int64_t D, int64_t capacity, int64_t budget) {
    return 2 * B * heads * move_parts(D, capacity, budget);
}

hipError_t launch_cache_evict(const EvictArgs &a, hipStream_t s) {
    const unsigned n = (unsigned)(a.c.B * a.c.heads);
    const int64_t capacity = (int64_t)a.c.width << a.c.page_log2;
    if (capacity <= kSelect) hipLaunchKernelGGL(k_evict_select<1>, dim3(n), dim3(kSelect), 0, s, a);
    else if (capacity <= 4 * kSelect) hipLaunchKernelGGL(k_evict_select<4>, dim3(n), dim3(kSelect), 0, s, a);
    else if (capacity <= 16 * kSelect) hipLaunchKernelGGL(k_evict_select<16>, dim3(n), dim3(kSelect), 0, s, a);
    else hipLaunchKernelGGL(k_evict_select<0>, dim3(n), dim3(kSelect), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.to == a.c.table) {
        hipLaunchKernelGGL((k_evict_move<true, 1024>), dim3(2 * n), dim3(1024), 0, s, a, 1);
        return hipGetLastError();
    }
    // (four chunks a workgroup: 54.5 us against 51.5 for 16 x 9000 -> 4096 entries, 69 against 73 for 8 x 16000 -> 12000)
    const int parts = (int)move_parts(a.c.D, capacity, a.budget);
    hipLaunchKernelGGL((k_evict_move<false, kMove>), dim3(2 * n * (unsigned)parts), dim3(kMove), 0, s, a, parts);
    return hipGetLastError();
}

}  // namespace qmm
