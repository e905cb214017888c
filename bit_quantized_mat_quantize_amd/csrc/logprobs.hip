// logprobs.hip -- log probabilities of given tokens, entropy and the most likely
// tokens of rows of logits (gfx950).  With z_i = scale * x_i over the allowed i:
//
//     m = max x,  S = sum_i e^{scale (x_i - m)},  T = sum_i scale (x_i - m) e^{scale (x_i - m)}
//     log p_i = scale (x_i - m) - log S,          H = log S - T / S
//
// One pass over the logits: each lane keeps a running (m, S, T) in fp32, S with
// what its rounding leaves, and rescales it when its maximum grows; exponents are
// taken in base 2; lanes, wavefronts and splits are joined in 64 bits.  T's terms
// are all <= 0, so the entropy has no cancellation.
//
// The k best ride in the same pass.  A token's key is 64 bits, the order of its
// logit above the complement of its index: keys are unique, and of equal logits
// the lower index is the larger key.  Each wavefront appends the keys that reach
// a common lower bound of the k-th best to a list in LDS.  The bound is the k-th
// largest of 64 (or 256) maxima, each over some of the threads: values that are all
// present.  It is taken after batches 1, 3, 9, 33, ... of a workgroup, so that the
// lists grow slowly; a list that is full all the same (equal or ascending logits)
// is cut back to its k best.  Both find the k-th largest by bisection over the bits:
// each step is a ballot and a count, no data moves.  At the end the lists of the
// workgroup are ranked by counting.
//
// A row is split over workgroups where there are few rows (partial statistics
// and keys go to the workspace, k_logprobs_merge joins them); otherwise one
// workgroup takes a row and the workspace is not used.  The pass is bound by
// reading the logits, for few rows by the latency of the launches.
#include "qmm_device.h"
#include "qmm_launch.h"

namespace qmm {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;
constexpr int kBatch = 16;     // logits per thread and batch; twice as many where rows are few and whole
constexpr int kList = 256;     // keys a wavefront's list holds
constexpr int kMaxK = 64;      // a cut leaves at most kMaxK, and 64 may be appended at once
constexpr int kMaxSplits = 64;
constexpr float kLn2 = 0.693147180559945309f;
constexpr float kLog2e = 1.44269504088896341f;
constexpr float kInf = __builtin_inff();

struct BF16 {
    uint16_t b;
};
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float to_f32(BF16 v) { return __uint_as_float((uint32_t)v.b << 16); }

// the logits of a 16-byte piece
template <typename T>
__device__ __forceinline__ void unpack(uint4 p, float (&y)[16 / sizeof(T)]) {
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            y[i] = __uint_as_float(w[i]);
        } else {
            const uint16_t h[2] = {(uint16_t)w[i], (uint16_t)(w[i] >> 16)};
            y[2 * i] = to_f32(__builtin_bit_cast(T, h[0]));
            y[2 * i + 1] = to_f32(__builtin_bit_cast(T, h[1]));
        }
    }
}

// ---- keys.  order(x) is monotone in x, and order(lowest finite) > 0; a key of 0 is no token.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);  // -0 and 0 are equal
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t o) {
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) {
    return ((uint64_t)order_of(x) << 32) | (uint32_t)~index;
}
// the smallest logit whose key can be >= key: the bound of the cheap test
__device__ __forceinline__ float value_bound(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return o < 0x00800000u ? -__FLT_MAX__ : of_order(o);  // below the order of the lowest finite number
}

__device__ __forceinline__ int lanes_below(uint64_t ballot) {
    return __builtin_amdgcn_mbcnt_hi((uint32_t)(ballot >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)ballot, 0));
}
// LDS that one wavefront writes and reads itself
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The largest bound that at least k of the wavefront's n * 64 values reach
// (0 if fewer than k are non-zero), stopping early at one that exactly k reach.
template <typename U, int n>
__device__ __forceinline__ U kth_bound(const U (&v)[n], int k) {
    U bound = 0;
#pragma unroll 1
    for (int bit = (int)sizeof(U) * 8 - 1; bit >= 0; --bit) {
        const U next = bound | (U(1) << bit);
        int c = 0;
#pragma unroll
        for (int i = 0; i < n; ++i) c += __popcll(__ballot(v[i] >= next));
        if (c >= k) bound = next;
        if (c == k) break;
    }
    return bound;
}

// One wavefront's candidates.
struct List {
    uint64_t *keys;  // LDS [kList]
    int count, k;
    uint64_t bound;  // no key below it can be among the k best
    float least;     // value_bound(bound)

    __device__ __forceinline__ void raise(uint64_t b) {
        if (b > bound) {
            bound = b;
            least = value_bound(b);
        }
    }
    // keep the k best (in any order)
    __device__ __forceinline__ void cut() {
        if (count <= k) return;
        const int lane = threadIdx.x & 63;
        uint64_t v[kList / kWave];
#pragma unroll
        for (int i = 0; i < kList / kWave; ++i) v[i] = i * kWave + lane < count ? keys[i * kWave + lane] : 0;
        const uint64_t b = kth_bound(v, k);
        int n = 0;
#pragma unroll
        for (int i = 0; i < kList / kWave; ++i) {
            const bool in = v[i] >= b;
            const uint64_t who = __ballot(in);
            if (in) keys[n + lanes_below(who)] = v[i];
            n += __popcll(who);
        }
        wave_lds_fence();
        count = n;
        raise(b);
    }
    // append the keys of the lanes that have one (all 64 lanes call it)
    __device__ __forceinline__ void add(uint64_t key, bool has) {
        uint64_t who = __ballot(has && key >= bound);
        if (who == 0) return;
        if (count + __popcll(who) > kList) {
            cut();
            who = __ballot(has && key >= bound);
        }
        if (who >> (threadIdx.x & 63) & 1) keys[count + lanes_below(who)] = key;
        wave_lds_fence();
        count += __popcll(who);
    }
};

// The order of the k-th largest of 64 * G maxima over the workgroup's threads, each
// over kWaves / G threads (0: fewer than k of them have a logit): at least k logits
// are not below it.
template <int G>
__device__ __forceinline__ uint32_t common_bound_of(int k, uint32_t (*lds)[kWave]) {
    uint32_t best[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
        best[g] = 0;
#pragma unroll
        for (int w = g; w < kWaves; w += G) {
            const uint32_t v = lds[w][threadIdx.x & 63];
            best[g] = v > best[g] ? v : best[g];
        }
    }
    __syncthreads();
    return kth_bound(best, k);
}
__device__ __forceinline__ uint32_t common_bound(uint32_t mine, int k, uint32_t (*lds)[kWave]) {
    lds[threadIdx.x >> 6][threadIdx.x & 63] = mine;
    __syncthreads();
    // of 8192 logits about 64 ln(64 / (64 - k)) reach the bound of 64 maxima: 24 for
    // k = 20, but 300 for k = 64, where four times as many maxima let 74 pass
    return k <= 20 ? common_bound_of<1>(k, lds) : common_bound_of<4>(k, lds);
}

// ---- running statistics in base 2: c = scale * log2(e)
// S is 1 plus what the other tokens have, often little: joins add in 64 bits, and
// log S is taken of S - 1.
template <int kCtrl>
__device__ __forceinline__ double dpp_f64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)dpp_i32<kCtrl>((int)(uint32_t)u), hi = (uint32_t)dpp_i32<kCtrl>((int)(u >> 32));
    return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_sum_f64(double v) {
    v += dpp_f64<0xB1>(v);
    v += dpp_f64<0x4E>(v);
    v += dpp_f64<0x141>(v);
    v += dpp_f64<0x140>(v);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < kWave; i += 16) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, i);
        const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), i);
        sum += __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
    }
    return sum;
}
struct Stats {
    float m, t;
    double s;
    // the same sums against a maximum to >= m
    __device__ __forceinline__ void rescale(float to, float c) {
        if (m == -kInf) {  // s and t are 0, or NaN, and stay so
            m = to;
            return;
        }
        const float d = (m - to) * c;
        const float f = __builtin_amdgcn_exp2f(d);
        t = f > 0.f ? f * (t + d * (float)s) : f * t;
        s *= f;
        m = to;
    }
    __device__ __forceinline__ void join_wave(float c) {
        rescale(wave_max(m), c);
        s = wave_sum_f64(s);
        t = wave_sum(t);
    }
    __device__ __forceinline__ bool none() const { return m == -kInf && s == 0.0; }  // nothing allowed, or all -inf
    __device__ __forceinline__ float log_s() const { return log1pf((float)(s - 1.0)); }
    // log p of logit x, in natural units throughout (the lowest finite logit times
    // log2(e) would overflow)
    __device__ __forceinline__ float logprob(float x, float scale) const {
        return none() ? -kInf : (x - m) * scale - log_s();
    }
    __device__ __forceinline__ float entropy() const { return none() ? 0.f : log_s() - t / (float)s * kLn2; }
};
// A thread's share: s + rest is the sum, rest what rounding left.
struct Share {
    float m, s, rest, t;
    __device__ __forceinline__ void rescale(float to, float c) {
        if (m != -kInf) {
            const float d = (m - to) * c;
            const float f = __builtin_amdgcn_exp2f(d);
            t = f > 0.f ? f * (t + d * s) : f * s;
            s = f * s;
            rest = f * rest;
        }
        m = to;
    }
    __device__ __forceinline__ void add(float bs, float bt) {
        const float sum = s + bs, b = sum - s;
        rest += (s - (sum - b)) + (bs - b);
        s = sum;
        t += bt;
    }
    __device__ __forceinline__ Stats stats() const { return Stats{m, t, (double)s + (double)rest}; }
};

__device__ __forceinline__ bool allowed(const uint32_t *mask, int i) { return mask[i >> 5] >> (i & 31) & 1; }

// ---- keys of the workgroup, at most one per thread, ranked: f(rank, key) for the
// k best, in any order.  Every thread calls it; returns the number of keys.
template <typename F>
__device__ __forceinline__ int rank_keys(uint64_t key, bool has, int k, uint64_t *all, int *counts, F f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint64_t who = __ballot(has);
    if (lane == 0) counts[wave] = __popcll(who);
    __syncthreads();
    int at = lanes_below(who), n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        at += w < wave ? counts[w] : 0;
        n += counts[w];
    }
    if (has) all[at] = key;
    __syncthreads();
    int rank = 0;
#pragma unroll 8
    for (int i = 0; i < n; ++i) rank += all[i] > key;
    if (has && rank < k) f(rank, key);
    return n;
}

// ---- results of one row.  A thread's first given token and its logit are
// fetched before the statistics are known.
struct Given {
    float x;
    bool valid;
};
template <typename T>
__device__ __forceinline__ Given given_token(const LogprobArgs &a, int64_t row, int64_t i) {
    Given g{-kInf, false};
    if (i < a.G) {
        const int tok = a.tokens[row * a.G + i];
        g.valid = tok >= 0 && tok < a.V;
        if (g.valid && (a.mask == nullptr || allowed(a.mask + row * a.mask_ld, tok)))
            g.x = to_f32(static_cast<const T *>(a.logits)[row * a.ld + tok]);
    }
    return g;
}
template <typename T>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, const Stats &st, int64_t row, Given g, uint64_t key,
                                           bool has, uint64_t *all, int *counts) {
    if (a.entropy != nullptr && threadIdx.x == 0) a.entropy[row] = st.entropy();
    for (int64_t i = threadIdx.x; i < a.G; i += kThreads) {
        if (i >= kThreads) g = given_token<T>(a, row, i);
        a.token_logprobs[row * a.G + i] = g.valid ? st.logprob(g.x, a.scale) : __builtin_nanf("");
    }
    if (a.k > 0) {
        int32_t *ids = a.top_ids + row * a.k;
        float *lps = a.top_logprobs + row * a.k;
        const int n = rank_keys(key, has, (int)a.k, all, counts, [&](int rank, uint64_t best) {
            ids[rank] = (int32_t)~(uint32_t)best;
            lps[rank] = st.logprob(of_order((uint32_t)(best >> 32)), a.scale);
        });
        for (int i = n + (int)threadIdx.x; i < a.k; i += kThreads) {  // fewer than k tokens are above -inf
            ids[i] = -1;
            lps[i] = -kInf;
        }
    }
}

// ---- the pass.  Workgroup = (row, split).  A row's whole 16-byte pieces,
// counted from the 16-byte boundary at or below its start, are divided among the
// splits; the up to 14 logits before the first and behind the last (rows need
// not start or end on a boundary) are a batch of their own in split 0.
//
// Measured: 1024 rows of 128256 fp32 logits, k = 1: 94 us, 5.6 TB/s, what a copy
// reaches; 513 rows of 50257 fp16 logits, k = 8: 23 us for 52 MB: about 50 cycles of
// vector instructions per 64 logits (an exponential is 16 of them), two rows per CU
// and three on one, and 6 us for the bounds and lists (17 us with k = 0); 32 rows of
// 128256 under masks, k = 20: 10.3 us in 16 splits each; one row of 32000, k = 5: 8.8
// us, of which the statistics take 5.5 and the bound and the ranking the rest.
template <typename T, bool MASK, int BATCH>
__global__ __launch_bounds__(kThreads) void k_logprobs(const LogprobArgs a, int splits) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int U = BATCH / VEC;  // pieces per thread and batch
    __shared__ uint64_t lists[kWaves][kList];
    __shared__ uint64_t all[kThreads];
    __shared__ int counts[kWaves];
    __shared__ uint32_t maxima[kWaves][kWave];
    __shared__ Stats wave_stats[kWaves];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x / (uint32_t)splits;
    const int split = (int)(blockIdx.x % (uint32_t)splits);
    const float c = a.scale * kLog2e;
    const int V = (int)a.V;
    const int64_t first = row * a.ld;
    const int lead = (int)(first % VEC);  // elements between the boundary and the row's start
    const T *x = static_cast<const T *>(a.logits) + (first - lead);
    const uint32_t *mask = MASK ? a.mask + row * a.mask_ld : nullptr;
    Given given{-kInf, false};
    if (splits == 1) given = given_token<T>(a, row, threadIdx.x);

    const int f0 = lead > 0 ? 1 : 0, f1 = (lead + V) / VEC;  // the whole pieces
    const int whole = f1 > f0 ? f1 - f0 : 0;
    const int per = (whole + splits - 1) / splits;
    const int j0 = f0 + split * per, j1 = j0 + per < f0 + whole ? j0 + per : f0 + whole;
    const int head = whole > 0 ? f0 * VEC - lead : V;  // logits [0, head) and [tail, V) are in no whole piece
    const int tail = whole > 0 ? f1 * VEC - lead : V;
    const bool edges = split == 0 && head + V - tail > 0;

    Share mine{-kInf, 0.f, 0.f, 0.f};
    List l{lists[wave], 0, (int)a.k, 0, -__FLT_MAX__};
    const int batches = (j1 - j0 + kThreads * U - 1) / (kThreads * U);
    for (int it = 0; it < batches + (edges ? 1 : 0); ++it) {
        float v[BATCH];
        int index0;      // of v[0]; v[u * VEC + q] follows at u * kThreads * VEC + q
        int filled = 1;  // pieces per thread with anything in them: a split's last batch is seldom full
        if (it < batches) {
            const int jt = j0 + it * kThreads * U + (int)threadIdx.x;
            index0 = jt * VEC - lead;
            filled = (j1 - (jt - (int)threadIdx.x) + kThreads - 1) / kThreads;
            uint4 p[U];
            uint32_t bits[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {  // pieces past the split's end read its last one
                const int at = jt + u * kThreads < j1 ? jt + u * kThreads : j1 - 1;
                p[u] = ld16(x + (int64_t)at * VEC);
                if (MASK) {
                    const int i = at * VEC - lead;
                    const uint32_t w0 = mask[i >> 5], w1 = mask[(i + VEC - 1) >> 5];
                    bits[u] = (uint32_t)((((uint64_t)w1 << 32) | w0) >> (i & 31));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const bool in = jt + u * kThreads < j1;
                float y[VEC];
                unpack<T>(p[u], y);
#pragma unroll
                for (int q = 0; q < VEC; ++q)
                    v[u * VEC + q] = !MASK || (in && (bits[u] >> q & 1)) ? y[q] : -kInf;
            }
            // behind the split's end, in its last batch (all the others do without: 700
            // rows of 128256 bf16 logits 51.0 -> 47.2 us)
            if (!MASK && j1 - (jt - (int)threadIdx.x) < kThreads * U) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < VEC; ++q) v[u * VEC + q] = jt + u * kThreads < j1 ? v[u * VEC + q] : -kInf;
            }
        } else {
            index0 = (int)threadIdx.x < head ? (int)threadIdx.x : tail + (int)threadIdx.x - head;
#pragma unroll
            for (int i = 0; i < BATCH; ++i) v[i] = -kInf;
            if (index0 < V && (!MASK || allowed(mask, index0))) v[0] = to_f32(x[lead + index0]);
        }

        float top = -kInf;
#pragma unroll
        for (int i = 0; i < BATCH; ++i) top = fmaxf(top, v[i]);
        if (top > mine.m) mine.rescale(top, c);
        // all of them -inf so far: any finite number in the maximum's place gives e = 0
        const float m = mine.m == -kInf ? 0.f : mine.m;
        // the batch's terms by themselves first, in two sums: next to the term of the
        // maximum each small one would be rounded at its size
        float bs[2] = {0.f, 0.f}, bt[2] = {0.f, 0.f};
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (u > 0 && u >= filled) break;
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float d = (v[u * VEC + q] - m) * c;
                const float e = __builtin_amdgcn_exp2f(d);
                bs[q % 2] += e;
                bt[q % 2] = __builtin_fmaf(fmaxf(d, -1.0e4f), e, bt[q % 2]);  // e is 0 there: keeps -inf * 0 out
            }
        }
        mine.add(bs[0] + bs[1], bt[0] + bt[1]);

        // after batches 1, 3, 9, 33, ...: after 1, 2, 3, 5, 9 it cost more than it saved
        // (513 rows of 50257, k = 8: 25.9 against 24.4 us), after 1, 5, 17 less than it
        // let through (27.3 us)
        if (a.k > 0 && (it == 0 || ((it & (it - 1)) == 0 && (it & 0x2aaaaaaa) != 0)))
            l.raise((uint64_t)common_bound(mine.m > -kInf ? order_of(mine.m) : 0, l.k, maxima) << 32);
        if (a.k > 0 && __ballot(top >= l.least) != 0) {
            uint32_t left = 0;  // which of this lane's logits may enter
#pragma unroll
            for (int i = BATCH - 1; i >= 0; --i) left = left + left + (v[i] >= l.least ? 1u : 0u);
            while (__ballot(left != 0) != 0) {
                const int i = left != 0 ? __builtin_ctz(left) : 0;
                float y = v[0];
#pragma unroll
                for (int q = 1; q < BATCH; ++q) y = i == q ? v[q] : y;
                l.add(key_of(y, (uint32_t)(index0 + i / VEC * (kThreads * VEC) + i % VEC)), left != 0);
                left &= left - 1;
            }
        }
    }
    if (l.count > kWave) l.cut();
    Stats st = mine.stats();
    st.join_wave(c);
    if (lane == 0) wave_stats[wave] = st;
    __syncthreads();
    st = lane < kWaves ? wave_stats[lane] : Stats{-kInf, 0.f, 0.0};
    st.join_wave(c);

    const bool has = lane < l.count;
    const uint64_t key = has ? l.keys[lane] : 0;
    if (splits == 1) {
        finish_row<T>(a, st, row, given, key, has, all, counts);
        return;
    }
    const int64_t part = row * splits + split;
    if (threadIdx.x == 0) {
        const uint64_t u = __builtin_bit_cast(uint64_t, st.s);
        a.ws_stats[part] = make_float4(st.m, st.t, __uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32)));
    }
    if (a.k > 0) {
        uint64_t *out = a.ws_keys + part * a.k;
        const int n = rank_keys(key, has, (int)a.k, all, counts, [&](int rank, uint64_t best) { out[rank] = best; });
        for (int i = n + (int)threadIdx.x; i < a.k; i += kThreads) out[i] = 0;
    }
}

// ---- the splits of a row joined: one workgroup per row.  32 rows of 16 splits and 20
// keys each: 5.8 us, the latency of a launch, of one load per thread, a bound and a
// ranking.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs_merge(const LogprobArgs a, int splits) {
    __shared__ uint64_t lists[kWaves][kList];
    __shared__ uint64_t all[kThreads];
    __shared__ int counts[kWaves];
    __shared__ uint32_t maxima[kWaves][kWave];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    const float c = a.scale * kLog2e;
    const Given given = given_token<T>(a, row, threadIdx.x);
    const int total = splits * (int)a.k;
    const uint64_t *in = a.ws_keys + row * total;
    Stats st{-kInf, 0.f, 0.0};
    if (lane < splits) {
        const float4 p = a.ws_stats[row * splits + lane];
        const uint64_t u = ((uint64_t)__float_as_uint(p.w) << 32) | __float_as_uint(p.z);
        st = Stats{p.x, p.y, __builtin_bit_cast(double, u)};
    }
    st.join_wave(c);
    constexpr int n = kMaxSplits * kMaxK / kThreads;  // keys per thread
    List l{lists[wave], 0, (int)a.k, 0, -__FLT_MAX__};
    if (a.k > 0) {
        uint64_t v[n], best = 0;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int at = i * kThreads + (int)threadIdx.x;
            v[i] = at < total ? in[at] : 0;
            best = v[i] > best ? v[i] : best;
        }
        l.raise((uint64_t)common_bound((uint32_t)(best >> 32), l.k, maxima) << 32);
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i * kThreads < total) l.add(v[i], v[i] != 0);
        if (l.count > kWave) l.cut();
    }
    const bool has = lane < l.count;
    const uint64_t key = has ? l.keys[lane] : 0;
    finish_row<T>(a, st, row, given, key, has, all, counts);
}

// A row of up to four batches (eight where 128 rows or more keep the CUs busy) is
// not split: 32000 logits, k = 5, take one workgroup 8.9 us, four of them 9.4 us with
// the second launch, which costs the caller another 4 us; 128 rows of 50257, k = 8:
// 16 us in one launch, 18 us in two.  Longer rows make two workgroups per CU (64 rows
// of 128256, k = 20, masked: 19.9 us with eight splits, 22.5 us with sixteen), and
// from 256 rows on one workgroup each (256 rows of 50257, k = 8: 16.3 us, 24.2 us in
// four; 400 of 128256: 44.9 us, 53.5 us in two).
int splits_of(int64_t M, int64_t V) {
    constexpr int64_t batch = kThreads * kBatch;
    if (M >= 256 || V <= (M < 128 ? 4 : 8) * batch) return 1;
    const int64_t s = 512 / M, most = (V + batch - 1) / batch;
    return (int)(s > most ? (most > kMaxSplits ? kMaxSplits : most) : (s > kMaxSplits ? kMaxSplits : s));
}

// A workgroup that has a row and a CU to itself waits for its loads more than it
// computes: it takes 32 logits per thread and batch (one row of 32000, k = 5: 10.9 -> 9.4
// us, 256 masked rows of 128256, k = 20: 44.8 -> 39.9 us, three sets of inputs in turn;
// 38.1 -> 35.1 us where the 256 MB cache holds the one set).  Where others run
// beside it or its part is short, 16 are faster (513 rows of 50257: 23.8 us, 25.8 us
// with 32; 32 rows of 128256 in 16 parts: 14.6 us, 15.3 us; 32 rows of 5000, less than
// one batch: 6.8 us, 7.3 us).
template <typename T, bool MASK>
void pass(const LogprobArgs &a, int splits, hipStream_t s) {
    const dim3 grid((unsigned)(a.M * splits));
    if (splits == 1 && a.M <= 256 && a.V > kThreads * kBatch)
        hipLaunchKernelGGL((k_logprobs<T, MASK, 2 * kBatch>), grid, dim3(kThreads), 0, s, a, splits);
    else
        hipLaunchKernelGGL((k_logprobs<T, MASK, kBatch>), grid, dim3(kThreads), 0, s, a, splits);
}

template <typename T>
hipError_t both(const LogprobArgs &a, hipStream_t s) {
    const int splits = splits_of(a.M, a.V);
    if (a.mask != nullptr) pass<T, true>(a, splits, s);
    else pass<T, false>(a, splits, s);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1) return e;
    hipLaunchKernelGGL(k_logprobs_merge<T>, dim3((unsigned)a.M), dim3(kThreads), 0, s, a, splits);
    return hipGetLastError();
}

}  // namespace

int64_t logprobs_max_k() { return kMaxK; }
int logprobs_splits(int64_t M, int64_t V) { return splits_of(M, V); }
int64_t logprobs_max_rows() { return (int64_t(1) << 32) / kThreads - 1; }

int64_t logprobs_workspace_bytes(int64_t M, int64_t V, int64_t k) {
    const int64_t splits = splits_of(M, V);
    return splits == 1 ? 0 : M * splits * (16 + 8 * k);
}

hipError_t launch_logprobs(int type, LogprobArgs a, void *ws, hipStream_t s) {
    const int64_t splits = splits_of(a.M, a.V);
    if (splits > 1) {
        a.ws_stats = static_cast<float4 *>(ws);
        a.ws_keys = reinterpret_cast<uint64_t *>(a.ws_stats + a.M * splits);
    }
    switch (type) {
        case 0: return both<float>(a, s);
        case 1: return both<_Float16>(a, s);
        default: return both<BF16>(a, s);
    }
}

}  // namespace qmm
