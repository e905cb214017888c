// logprobs.hip -- log probabilities of given tokens, entropy and the most likely
// tokens of rows of logits (gfx950).  With z_i = scale * x_i over the allowed i:
//
//     m = max x,  S = sum_i e^{scale (x_i - m)},  T = sum_i scale (x_i - m) e^{scale (x_i - m)}
//     log p_i = scale (x_i - m) - log S,          H = log S - T / S
//
// One pass over the logits: each lane keeps a running (m, S, T) in fp32 and
// rescales it when its maximum grows; exponents are taken in base 2.  T's terms
// are all <= 0, so the entropy has no cancellation.
//
// The k best ride in the same pass.  A token's key is 64 bits, the order of its
// logit above the complement of its index: keys are unique, and of equal logits
// the lower index is the larger key.  Each wavefront keeps a lower bound of its
// k-th best and appends what is not below it to a list in LDS.  The first bound
// comes from the lanes' maxima of the first batch (the k-th largest of 64 values
// that are all present); a full list is cut back to its k best, which raises the
// bound, so after a few thousand logits hardly any pass and a batch costs one
// comparison.  Both cuts find the k-th largest by bisection over the bits: each
// step is a ballot and a count, no data moves.  At the end the lists of the
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

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
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

// ---- running statistics in base 2: c = scale * log2(e)
struct Stats {
    float m, s, t;
    // the same sums against a maximum to >= m
    __device__ __forceinline__ void rescale(float to, float c) {
        if (m == -kInf) {  // s and t are 0, or NaN, and stay so
            m = to;
            return;
        }
        const float d = (m - to) * c;
        const float f = __builtin_amdgcn_exp2f(d);
        t = f > 0.f ? f * (t + d * s) : f * s;
        s = f * s;
        m = to;
    }
    __device__ __forceinline__ void join(Stats o, float c) {
        const float to = fmaxf(m, o.m);
        rescale(to, c);
        o.rescale(to, c);
        s += o.s;
        t += o.t;
    }
    __device__ __forceinline__ void join_wave(float c) {
        rescale(wave_max(m), c);
        s = wave_sum(s);
        t = wave_sum(t);
    }
    // log p of logit x, in natural units throughout (the lowest finite logit times
    // log2(e) would overflow); an empty row (nothing allowed, or all -inf) has none
    __device__ __forceinline__ float logprob(float x, float scale) const {
        if (m == -kInf && s == 0.f) return -kInf;
        return (x - m) * scale - log2f(s) * kLn2;
    }
    __device__ __forceinline__ float entropy() const {
        if (m == -kInf && s == 0.f) return 0.f;
        return (log2f(s) - t / s) * kLn2;
    }
};

__device__ __forceinline__ bool allowed(const uint32_t *mask, int i) { return mask[i >> 5] >> (i & 31) & 1; }

// ---- the workgroup's lists, ranked: f(rank, key) for the k best, in any order.
// Every thread calls it; lists hold at most k keys each (k <= 64).
template <typename F>
__device__ __forceinline__ int rank_lists(const List &l, uint64_t *all, int *counts, F f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (lane == 0) counts[wave] = l.count;
    const uint64_t key = lane < l.count ? l.keys[lane] : 0;
    __syncthreads();
    int off = 0, n = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        off += w < wave ? counts[w] : 0;
        n += counts[w];
    }
    if (lane < l.count) all[off + lane] = key;
    __syncthreads();
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += all[i] > key;
    if (lane < l.count && rank < l.k) f(rank, key);
    return n;
}

// ---- results of one row
__device__ __forceinline__ void finish_row(const LogprobArgs &a, const Stats &st, int64_t row, const List &l,
                                           uint64_t *all, int *counts) {
    const bool any = !(st.m == -kInf && st.s == 0.f);
    if (a.entropy != nullptr && threadIdx.x == 0) a.entropy[row] = st.entropy();
    if (a.k > 0) {
        int32_t *ids = a.top_ids + row * a.k;
        float *lps = a.top_logprobs + row * a.k;
        const int n = rank_lists(l, all, counts, [&](int rank, uint64_t key) {
            ids[rank] = (int32_t)~(uint32_t)key;
            lps[rank] = st.logprob(of_order((uint32_t)(key >> 32)), a.scale);
        });
        for (int i = n + (int)threadIdx.x; i < a.k; i += kThreads) {  // fewer than k tokens have a probability
            ids[i] = -1;
            lps[i] = any && st.s != st.s ? st.s : -kInf;
        }
    }
}
template <typename T>
__device__ __forceinline__ void given_tokens(const LogprobArgs &a, const Stats &st, int64_t row) {
    const T *x = static_cast<const T *>(a.logits) + row * a.ld;
    const uint32_t *mask = a.mask != nullptr ? a.mask + row * a.mask_ld : nullptr;
    for (int64_t i = threadIdx.x; i < a.G; i += kThreads) {
        const int tok = a.tokens[row * a.G + i];
        float lp = __builtin_nanf("");
        if (tok >= 0 && tok < a.V)
            lp = st.logprob(mask == nullptr || allowed(mask, tok) ? to_f32(x[tok]) : -kInf, a.scale);
        a.token_logprobs[row * a.G + i] = lp;
    }
}

// ---- the pass.  Workgroup = (row, split); a split is a range of 16-byte pieces
// of the row, counted from the 16-byte boundary at or below the row's start.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs(const LogprobArgs a, int splits) {
    constexpr int VEC = 16 / sizeof(T);
    constexpr int U = 16 / VEC;  // pieces per thread and batch: 16 logits
    __shared__ uint64_t lists[kWaves][kList];
    __shared__ uint64_t all[kWaves * kMaxK];
    __shared__ int counts[kWaves];
    __shared__ Stats wave_stats[kWaves];
    struct alignas(16) Pack {
        T e[VEC];
    };

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x / (uint32_t)splits;
    const int split = (int)(blockIdx.x % (uint32_t)splits);
    const float c = a.scale * kLog2e;
    const int V = (int)a.V;
    const int64_t first = row * a.ld;
    const int lead = (int)(first % VEC);  // elements between the boundary and the row's start
    const T *x = static_cast<const T *>(a.logits) + (first - lead);
    const uint32_t *mask = a.mask != nullptr ? a.mask + row * a.mask_ld : nullptr;
    const int pieces = (lead + V + VEC - 1) / VEC;
    const int per = (pieces + splits - 1) / splits;
    const int j0 = split * per, j1 = j0 + per < pieces ? j0 + per : pieces;

    Stats st{-kInf, 0.f, 0.f};
    List l{lists[wave], 0, (int)a.k, 0, -__FLT_MAX__};
    for (int jb = j0; jb < j1; jb += kThreads * U) {
        float v[U * VEC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int j = jb + u * kThreads + threadIdx.x;
            const int i0 = j * VEC - lead;  // index of the piece's first logit
#pragma unroll
            for (int q = 0; q < VEC; ++q) v[u * VEC + q] = -kInf;
            if (j < j1) {
                if (i0 >= 0 && i0 + VEC <= V) {
                    const Pack p = *reinterpret_cast<const Pack *>(x + (int64_t)j * VEC);
                    uint32_t bits = ~0u;
                    if (mask != nullptr) {
                        const uint32_t w0 = mask[i0 >> 5], w1 = mask[(i0 + VEC - 1) >> 5];
                        bits = (uint32_t)((((uint64_t)w1 << 32) | w0) >> (i0 & 31));
                    }
#pragma unroll
                    for (int q = 0; q < VEC; ++q) v[u * VEC + q] = bits >> q & 1 ? to_f32(p.e[q]) : -kInf;
                } else {
#pragma unroll
                    for (int q = 0; q < VEC; ++q)
                        if (i0 + q >= 0 && i0 + q < V && (mask == nullptr || allowed(mask, i0 + q)))
                            v[u * VEC + q] = to_f32(x[(int64_t)j * VEC + q]);
                }
            }
        }
        float top = -kInf;
#pragma unroll
        for (int i = 0; i < U * VEC; ++i) top = fmaxf(top, v[i]);
        if (top > st.m) st.rescale(top, c);
        // all of them -inf so far: any finite number in the maximum's place gives e = 0
        const float m = st.m == -kInf ? 0.f : st.m;
        // the batch's terms by themselves first: next to the term of the maximum each
        // small one would be rounded at its size
        float bs = 0.f, bt = 0.f;
#pragma unroll
        for (int i = 0; i < U * VEC; ++i) {
            const float d = (v[i] - m) * c;
            const float e = __builtin_amdgcn_exp2f(d);
            bs += e;
            bt += fmaxf(d, -1.0e4f) * e;  // e is 0 there: keeps -inf * 0 out
        }
        st.s += bs;
        st.t += bt;
        if (a.k > 0) {
            if (jb == j0) {
                const uint32_t o[1] = {top > -kInf ? order_of(top) : 0};
                l.raise((uint64_t)kth_bound(o, l.k) << 32);
            }
            if (__ballot(top >= l.least) != 0) {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int q = 0; q < VEC; ++q) {
                        const float y = v[u * VEC + q];
                        if (__ballot(y >= l.least) != 0)
                            l.add(key_of(y, (uint32_t)((jb + u * kThreads + (int)threadIdx.x) * VEC - lead + q)),
                                  y >= l.least);
                    }
            }
        }
    }
    if (a.k > 0) l.cut();
    st.join_wave(c);
    if (lane == 0) wave_stats[wave] = st;
    __syncthreads();
    st = wave_stats[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) st.join(wave_stats[w], c);

    if (splits == 1) {
        finish_row(a, st, row, l, all, counts);
        given_tokens<T>(a, st, row);
        return;
    }
    const int64_t part = row * splits + split;
    if (threadIdx.x == 0) a.ws_stats[part] = make_float4(st.m, st.s, st.t, 0.f);
    if (a.k > 0) {
        uint64_t *out = a.ws_keys + part * a.k;
        const int n = rank_lists(l, all, counts, [&](int rank, uint64_t key) { out[rank] = key; });
        for (int i = n + (int)threadIdx.x; i < a.k; i += kThreads) out[i] = 0;
    }
}

// ---- the splits of a row joined: one workgroup per row
template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs_merge(const LogprobArgs a, int splits) {
    __shared__ uint64_t lists[kWaves][kList];
    __shared__ uint64_t all[kWaves * kMaxK];
    __shared__ int counts[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t row = blockIdx.x;
    const float c = a.scale * kLog2e;
    Stats st{-kInf, 0.f, 0.f};
    if (lane < splits) {
        const float4 p = a.ws_stats[row * splits + lane];
        st = Stats{p.x, p.y, p.z};
    }
    st.join_wave(c);
    List l{lists[wave], 0, (int)a.k, 0, -__FLT_MAX__};
    if (a.k > 0) {
        constexpr int n = kMaxSplits * kMaxK / kThreads;
        const int total = splits * (int)a.k;
        const uint64_t *in = a.ws_keys + row * total;
        uint64_t v[n], top[1] = {0};
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int at = i * kThreads + threadIdx.x;
            v[i] = at < total ? in[at] : 0;
            top[0] = v[i] > top[0] ? v[i] : top[0];
        }
        l.raise(kth_bound(top, l.k));
#pragma unroll
        for (int i = 0; i < n; ++i)
            if (i * kThreads < total) l.add(v[i], v[i] != 0);
        l.cut();
    }
    finish_row(a, st, row, l, all, counts);
    given_tokens<T>(a, st, row);
}

// enough workgroups to fill the chip (four per CU), each with at least 2048 logits
int splits_of(int64_t M, int64_t V) {
    int64_t s = (1024 + M - 1) / M;
    const int64_t most = (V + 2047) / 2048;
    s = s > most ? most : s;
    return (int)(s > kMaxSplits ? kMaxSplits : s);
}

template <typename T>
hipError_t both(const LogprobArgs &a, hipStream_t s) {
    const int splits = splits_of(a.M, a.V);
    hipLaunchKernelGGL(k_logprobs<T>, dim3((unsigned)(a.M * splits)), dim3(kThreads), 0, s, a, splits);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || splits == 1) return e;
    hipLaunchKernelGGL(k_logprobs_merge<T>, dim3((unsigned)a.M), dim3(kThreads), 0, s, a, splits);
    return hipGetLastError();
}

}  // namespace

int64_t logprobs_max_k() { return kMaxK; }
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
