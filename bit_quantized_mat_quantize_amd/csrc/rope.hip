// rope.hip -- rotary positions (gfx950): the pair (a, b) of a head at angle
// theta = position * frequency becomes m * (a cos theta - b sin theta,
// a sin theta + b cos theta).
//
// The frequency of pair i is base^(-2i/rot), over factors[i] where they are
// given, times 1 - r_i (1 - freq_scale) with r_i = clamp((i - low) / (high - low))
// (1 without a ramp).  The angle is formed in 64 bits, in turns, and cut to half a
// turn there: at a position of 10^6 fp32 would leave 0.06 of a radian.  Sine and
// cosine are rounded to fp32 once, the products and the sum are fp32.
//
// A workgroup forms one token's angles (one pair per thread, in LDS) and turns them
// into that token's heads, so the 64-bit work is paid once per token and not per
// head.  Everything else is 16-byte loads and stores: bound by HBM for prompts (4099
// tokens of 40 heads of 128 in bf16: 14.3 us, 5.9 TB/s, some of it from the caches), by
// the launch for single tokens, whose heads several workgroups share (40 heads of 128
// in fp32: 2.6 us).
#include "kv_device.h"

namespace qmm {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 1024;
constexpr int kUnits = 4;  // loads in flight per thread

template <int TYPE, int V>
__device__ __forceinline__ void load(const void *p, int64_t at, float *v) {
    if constexpr (V == 8) kv_load8<TYPE>(p, at, v);
    else if constexpr (V == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + at);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else if constexpr (TYPE == 0) v[0] = static_cast<const float *>(p)[at];
    else if constexpr (TYPE == 1) v[0] = f16_bits_to_f32(static_cast<const uint16_t *>(p)[at]);
    else v[0] = __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[at] << 16);
}
template <int TYPE, int V>
__device__ __forceinline__ void store(void *p, int64_t at, const float *v) {
    if constexpr (V == 8) kv_store8<TYPE>(p, at, v);
    else if constexpr (V == 4) *reinterpret_cast<float4 *>(static_cast<float *>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else if constexpr (TYPE == 0) static_cast<float *>(p)[at] = v[0];
    else static_cast<uint16_t *>(p)[at] = (uint16_t)(TYPE == 1 ? f32_to_f16_bits(v[0]) : bf16_bits(v[0]));
}

// V elements per access: 16 bytes, or 1 where sizes or strides are no multiples of them.
// A unit is V pairs (half layout), V elements of adjacent pairs (interleaved; one pair
// where V is 1) or V elements behind the rotated part, which are copied.
template <int TYPE, bool INTER, int V>
__global__ __launch_bounds__(kThreads) void k_rope(RopeArgs a, int share) {
    __shared__ float2 turn[kMaxDim / 2];
    const int64_t t = blockIdx.x / (unsigned)share;
    const int part = (int)(blockIdx.x - t * share), half = a.rot / 2;
    const double pos = (double)a.positions[t];
    for (int i = threadIdx.x; i < half; i += kThreads) {
        double f = exp2(-2.0 * i / a.rot * a.log2_base);
        if (a.factors != nullptr) f /= (double)a.factors[i];
        double r = 1.0;
        if (a.high > a.low) r = fmin(1.0, fmax(0.0, (i - a.low) / (a.high - a.low)));
        f *= 1.0 - r * (1.0 - a.freq_scale);
        double turns = pos * (f * 0.15915494309189533577);  // over 2 pi
        turns -= rint(turns);
        double s, c;
        sincospi(2.0 * turns, &s, &c);
        turn[i] = make_float2((float)(c * a.magnitude), (float)(s * a.magnitude));
    }
    __syncthreads();
    constexpr int PAIRS = INTER ? (V == 1 ? 1 : V / 2) : V;
    const int turned = half / PAIRS, copied = a.out == a.x ? 0 : (a.D - a.rot) / V;
    const int per_head = turned + copied, n = a.H * per_head;
    const int64_t x0 = t * a.ld_x, o0 = t * a.ld_out;
    for (int u0 = part * kThreads + threadIdx.x; u0 < n; u0 += share * kThreads * kUnits) {
        float v[kUnits][2 * V];
        int64_t from[kUnits], to[kUnits];
        int pair[kUnits], back[kUnits];  // first pair or -1 (copied); elements between the two halves of the unit
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            const int u = u0 + q * share * kThreads;
            if (u >= n) break;
            const int h = u / per_head, k = u - h * per_head;
            const bool copy = k >= turned;
            const int e = copy ? a.rot + (k - turned) * V : (INTER ? 2 : 1) * PAIRS * k;
            pair[q] = copy ? -1 : PAIRS * k;
            back[q] = copy || (INTER && V > 1) ? 0 : (INTER ? 1 : half);
            from[q] = x0 + h * a.head_x + e;
            to[q] = o0 + h * a.head_out + e;
            load<TYPE, V>(a.x, from[q], v[q]);
            if (back[q]) load<TYPE, V>(a.x, from[q] + back[q], v[q] + V);
        }
#pragma unroll
        for (int q = 0; q < kUnits; ++q) {
            if (u0 + q * share * kThreads >= n) break;
            if (pair[q] >= 0) {
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const int ia = INTER && V > 1 ? 2 * i : i, ib = INTER && V > 1 ? 2 * i + 1 : V + i;
                    const float2 cs = turn[pair[q] + i];
                    const float x = v[q][ia], y = v[q][ib];
                    v[q][ia] = fmaf(x, cs.x, -(y * cs.y));
                    v[q][ib] = fmaf(x, cs.y, y * cs.x);
                }
            }
            store<TYPE, V>(a.out, to[q], v[q]);
            if (back[q]) store<TYPE, V>(a.out, to[q] + back[q], v[q] + V);
        }
    }
}

template <int TYPE, bool INTER>
hipError_t launch(const RopeArgs &a, hipStream_t s) {
    constexpr int V = TYPE == 0 ? 4 : 8;
    const int64_t all = a.ld_x | a.ld_out | a.head_x | a.head_out | a.D | (INTER ? a.rot : a.rot / 2);
    const bool wide = all % V == 0;
    const int64_t units = (int64_t)a.H * (a.D / (wide ? V : 1));
    // a token's heads on several workgroups while there are few tokens (in a graph: one of 40 heads of 128 2.97 us, on one
    // workgroup 3.26; 64 3.18 and 3.50; 256 3.73 and 3.83)
    int64_t share = (units + kThreads - 1) / kThreads;
    const int64_t want = (2 * 256 + a.T - 1) / a.T;
    if (share > want) share = want;
    if (share < 1) share = 1;
    const dim3 grid((unsigned)(a.T * share));
    if (wide) hipLaunchKernelGGL((k_rope<TYPE, INTER, V>), grid, dim3(kThreads), 0, s, a, (int)share);
    else hipLaunchKernelGGL((k_rope<TYPE, INTER, 1>), grid, dim3(kThreads), 0, s, a, (int)share);
    return hipGetLastError();
}

}  // namespace

int64_t rope_max_dim() { return kMaxDim; }

hipError_t launch_rope(int type, bool interleaved, const RopeArgs &a, hipStream_t s) {
    if (type == 0) return interleaved ? launch<0, true>(a, s) : launch<0, false>(a, s);
    if (type == 1) return interleaved ? launch<1, true>(a, s) : launch<1, false>(a, s);
    return interleaved ? launch<2, true>(a, s) : launch<2, false>(a, s);
}

}  // namespace qmm
