// evict.hip -- a cache within its budget (gfx950): per sequence and head the newest
// entries and, of the others, those of the most accumulated weight, ties to the
// lower index; what stays moves together in its order.
//
// k_evict_select, one workgroup per (sequence, head): the weights' bits, mapped to
// unsigned keys of the same order, by radix select in digits of 11, 11 and 10 bits (a
// histogram in LDS each: integer counts, so their order does not matter), which gives the
// key of the last entry that stays and how many of its equals do; then each
// wavefront counts and writes its own range's places by ballots.
//
// k_evict_move, one workgroup per (sequence, head, keys or values): entries in
// ascending order, a chunk at a time, where all of a chunk is in registers before
// any of it is stored.  An entry only ever moves down, so chunks yet to be read lie
// above everything stored before: the pages may be the sequence's own.
#include "kv_device.h"

namespace qmm {
namespace {

constexpr int kSelect = 1024, kBins = 2048;
constexpr int kMove = 1024;

// larger keys for larger weights, -0 as 0, NaN above all
__device__ __forceinline__ uint32_t order_key(float m) {
    if (m != m) return 0xffffffffu;
    const uint32_t u = __float_as_uint(m + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ __launch_bounds__(kSelect) void k_evict_select(EvictArgs a) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t wave_above[kSelect / 64], wave_equal[kSelect / 64];
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
    for (int i = tid; i < a.recent; i += kSelect) {
        ids[need + i] = old + i;
        mass_out[need + i] = mass[old + i];
    }
    if (need == 0) return;
    uint32_t prefix = 0, left = need;  // the key's digits found so far; entries to take among those that share them
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
        for (int i = tid; i < kBins; i += kSelect) hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < old; i += kSelect) {
            const uint32_t key = order_key(mass[i]);
            if (pass == 0 || (key >> (shift + bits)) == prefix) atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1)], 1u);
        }
        __syncthreads();
        if (wave == 0) {  // from the largest digit down: lane i has the bins behind i * kBins / 64 of them
            constexpr int per = kBins / 64;
            uint32_t sum = 0;
            for (int i = 0; i < per; ++i) sum += hist[kBins - 1 - (lane * per + i)];
            uint32_t before = sum;
            for (int o = 1; o < 64; o <<= 1) {
                const uint32_t up = __shfl_up(before, o, 64);
                if (lane >= o) before += up;
            }
            before -= sum;
            if (before < left && before + sum >= left) {
                for (int i = 0; i < per; ++i) {
                    const int bin = kBins - 1 - (lane * per + i);
                    if (before + hist[bin] >= left) {
                        found[0] = bin;
                        found[1] = left - before;
                        break;
                    }
                    before += hist[bin];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << bits) | found[0];
        left = found[1];
        __syncthreads();
    }
    // entries above the key stay, and the first `left` of those that equal it
    const int per = ((old + kSelect - 1) / kSelect) * 64;  // positions of a wavefront
    const int p0 = wave * per, p1 = p0 + per < old ? p0 + per : old;
    uint32_t above = 0, equal = 0;
    for (int i = p0; i < p1; i += 64) {
        const uint32_t key = i + lane < p1 ? order_key(mass[i + lane]) : 0;
        const bool in = i + lane < p1;
        above += __popcll(__ballot(in && key > prefix));
        equal += __popcll(__ballot(in && key == prefix));
    }
    if (lane == 0) {
        wave_above[wave] = above;
        wave_equal[wave] = equal;
    }
    __syncthreads();
    uint32_t taken = 0, equals = 0;
    for (int w = 0; w < wave; ++w) {
        taken += wave_above[w];
        equals += wave_equal[w];
    }
    taken += equals < left ? equals : left;
    const uint64_t below = (uint64_t(1) << lane) - 1;
    for (int i = p0; i < p1; i += 64) {
        const bool in = i + lane < p1;
        const float m = in ? mass[i + lane] : 0.0f;
        const uint32_t key = order_key(m);
        const uint64_t eq = __ballot(in && key == prefix);
        const bool stays = in && (key > prefix || (key == prefix && equals + __popcll(eq & below) < left));
        const uint64_t all = __ballot(stays);
        if (stays) {
            const uint32_t at = taken + __popcll(all & below);
            ids[at] = i + lane;
            mass_out[at] = m;
        }
        taken += __popcll(all);
        equals += __popcll(eq);
    }
}

// a value that another thread's store may replace: read for good before the barrier
__device__ __forceinline__ void arrived(uint4 &v, uint32_t &s) {
    asm volatile("" : "+v"(v.x), "+v"(v.y), "+v"(v.z), "+v"(v.w), "+v"(s));
}

__global__ __launch_bounds__(kMove) void k_evict_move(EvictArgs a) {
    const int x = blockIdx.x, part = x & 1, h = (x >> 1) % a.c.heads, b = (x >> 1) / a.c.heads;
    const int D = a.c.D, nb = D / 32, lg = a.c.page_log2, mask = (1 << lg) - 1;
    const int32_t *ids = a.ids + ((int64_t)b * a.c.heads + h) * a.budget;
    const int32_t *to = a.to + (int64_t)b * a.to_width;
    const int most = a.c.width << lg, given = a.c.lens[b];
    const int L = given < 0 ? 0 : (given > most ? most : given), n = L < a.budget ? L : a.budget;
    const int chunk = kMove / nb & ~3;  // entries at a time: one 16-byte piece of codes and one scale per thread
    const int tid = threadIdx.x, words = D / 8;
    const bool active = tid < chunk * nb;
    // keys: piece p of entry j; values: word w of the entries 4g .. 4g + 3; scales: block s of entry i
    const int j = tid / nb, p = tid - j * nb, g = tid / words, w = tid - g * words, s = tid / chunk, i = tid - s * chunk;
    auto chunk_of = [&](int page) { return page >= 0 && page < a.c.pages ? kv_chunk(a.c, page, part, h) : nullptr; };
    auto source = [&](int at) -> const uint8_t * {  // of entry `at` of those that stay
        if (at >= n) return nullptr;
        return chunk_of(a.c.table[(int64_t)b * a.c.width + (ids[at] >> lg)]);
    };
    auto read = [&](int c0, uint4 &v, uint32_t &scale) {
        v = make_uint4(0, 0, 0, 0);
        scale = 0x7e00u;  // an entry whose page is not there is NaN
        if (!active) return;
        if (part == 0) {
            if (const uint8_t *q = source(c0 + j)) v = ld16(q + (ids[c0 + j] & mask) * (D / 2) + p * 16);
        } else {
            uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (const uint8_t *q = source(c0 + 4 * g + e))
                    u[e] = reinterpret_cast<const uint32_t *>(q)[kv_value_word(D, ids[c0 + 4 * g + e] & mask, w)];
            v = make_uint4(u[0], u[1], u[2], u[3]);
        }
        if (const uint8_t *q = source(c0 + i))
            scale = reinterpret_cast<const uint16_t *>(q)[kv_scale_at(a.c, ids[c0 + i] & mask, s)];
    };
    auto write = [&](int c0, const uint4 &v, uint32_t scale) {
        if (!active) return;
        if (part == 0) {
            const int at = c0 + j;
            if (uint8_t *q = at < n ? chunk_of(to[at >> lg]) : nullptr)
                *reinterpret_cast<uint4 *>(q + (at & mask) * (D / 2) + p * 16) = v;
        } else {
            const int at = c0 + 4 * g;
            if (uint8_t *q = at < n ? chunk_of(to[at >> lg]) : nullptr) {
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
        if (uint8_t *q = at < n ? chunk_of(to[at >> lg]) : nullptr)
            reinterpret_cast<uint16_t *>(q)[kv_scale_at(a.c, at & mask, s)] = (uint16_t)scale;
    };
    uint4 v, next;
    uint32_t scale, next_scale;
    read(0, v, scale);
    for (int c0 = 0; c0 < n; c0 += chunk) {
        read(c0 + chunk, next, next_scale);
        arrived(v, scale);
        __syncthreads();
        write(c0, v, scale);
        v = next;
        scale = next_scale;
    }
}

}  // namespace

hipError_t launch_cache_evict(const EvictArgs &a, hipStream_t s) {
    const unsigned n = (unsigned)(a.c.B * a.c.heads);
    hipLaunchKernelGGL(k_evict_select, dim3(n), dim3(kSelect), 0, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_evict_move, dim3(2 * n), dim3(kMove), 0, s, a);
    return hipGetLastError();
}

}  // namespace qmm
