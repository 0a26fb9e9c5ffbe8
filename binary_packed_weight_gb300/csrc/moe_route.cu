// moe_route.cu -- a mixture-of-experts router: scores, groups, top-k,
// renormalised weights, the plan (slots ordered by expert), and the gradient
// of the weights to the logits.
//
// A warp takes a token.  Lane i holds experts i*V .. i*V+V-1 in registers, so
// a row is read once in wide loads, the lowest lane that holds a maximum also
// holds the lowest expert, and the softmax sum's tree over neighbouring
// experts is V-1 additions in the lane and five shuffles.  Selection values
// are compared as order-preserving 32-bit keys: one redux.max and one ballot
// for each of the k experts.  A lane keeps its three best at hand and looks
// through its keys again only when it has won three times.
//
// The plan is a stable counting sort of the T*k slots.  Up to a few hundred
// tokens one cluster of CTAs does all of it, each CTA reading the others'
// counts through distributed shared memory.  Beyond, each CTA of the routing
// kernel leaves its chunk's counts, and a second kernel (its launch overlaps
// the first) turns them into each chunk's first positions and writes the slots.
// Within a chunk, warps count their 32 slots by match.any and a prefix over the
// warps orders them, so there is no atomic whose order could matter.
//
// Bound: a few tokens by the call (1x64: 7 us) and the latency of the picks (300x160
// in groups: 9.8).  Many (16384x256, 4 of 8 groups, top 8: 26.5 us): 998 warp instructions a
// token, a third of them the exact scores, are about 14 us of issue; the slots are 65 % busy,
// the rest waits in the chain of a pick (redux, ballot, shuffle) with one token a warp, and
// the plan's kernel is 6 to 7 of it.  The gradient's 16384x128 takes 6.5 us, of which the
// kernel 6.3 (in a replayed graph); 100x60 6.3 and 1.6.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "../../include/tq2.h"
#include "ptx.cuh"
#include "tq2_internal.h"

namespace tq2 {

namespace {

constexpr float ROUTE_TINY = 1.17549435e-38f;      // 2^-126
constexpr float ROUTE_MOST = 3.402823466e+38f;     // largest f32
constexpr int ROUTE_CLUSTER = 16;                  // CTAs of a cluster at most

struct RouteArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    int64_t T;
    int E, k, score, groups, top_groups, renorm;
    float scale;
    int32_t* ids;
    float* weights;
    int32_t* offsets;
    int32_t* slots;
    uint16_t* counts;                              // [chunks][E rounded up to even], two-kernel plan
    int64_t chunk;                                 // tokens of a CTA
    int vec;                                       // rows can be read in wide loads
    int gsize, gshift, gwhole;                     // groups: experts, log2 of the lanes; its lanes hold its experts
    int off_rows;                                  // groups: the warps' rows in shared memory (int index)
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// The widest word that V elements of T are whole words of.
template <int BYTES>
struct Word { using type = uint16_t; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<16> { using type = uint4; };
template <class T, int V>
struct Wide {
    static constexpr int BYTES = V * (int)sizeof(T) >= 16 ? 16 : V * (int)sizeof(T);
    using word = typename Word<BYTES>::type;
    static constexpr int WORDS = V * (int)sizeof(T) / BYTES;
};

// Experts lane*V .. of a row, -inf past its end.
template <class T, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, bool vec, float (&v)[V]) {
    const int e0 = lane * V;
    if (vec) {
        T raw[V];
        if (e0 < E) {
#pragma unroll
            for (int i = 0; i < Wide<T, V>::WORDS; ++i)
                reinterpret_cast<typename Wide<T, V>::word*>(raw)[i] =
                    reinterpret_cast<const typename Wide<T, V>::word*>(row + e0)[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) raw[i] = from_f32<T>(-INFINITY);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = to_f32(raw[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = e0 + i < E ? to_f32(row[e0 + i]) : -INFINITY;
    }
}
template <class T, int V>
__device__ __forceinline__ void store_row(T* row, int E, int lane, bool vec, const float (&v)[V]) {
    const int e0 = lane * V;
    if (vec) {
        if (e0 < E) {
            T raw[V];
#pragma unroll
            for (int i = 0; i < V; ++i) raw[i] = from_f32<T>(v[i]);
#pragma unroll
            for (int i = 0; i < Wide<T, V>::WORDS; ++i)
                reinterpret_cast<typename Wide<T, V>::word*>(row + e0)[i] =
                    reinterpret_cast<const typename Wide<T, V>::word*>(raw)[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e0 + i < E) row[e0 + i] = from_f32<T>(v[i]);
    }
}

// Available experts keep their logit (at most the largest f32), others get -inf.
__device__ __forceinline__ float available(float l, float bias) {
    return l > -INFINITY && bias > -INFINITY ? fminf(l, ROUTE_MOST) : -INFINITY;
}

// Row maximum and softmax sum of the available logits: neighbours first.
template <int V>
__device__ __forceinline__ float tree_sum(const float (&v)[V]) {
    float s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = v[i];
#pragma unroll
    for (int n = V; n > 1; n >>= 1)
#pragma unroll
        for (int i = 0; i < n / 2; ++i) s[i] = s[2 * i] + s[2 * i + 1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    return s[0];
}
__device__ __forceinline__ float warp_max(float m) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return m;
}
__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}
__device__ __forceinline__ float sigmoid(float l) { return __frcp_rn(1.0f + expf(-l)); }   // = 1 / (..), rounded

// Larger value, larger key (v is not -0: scores are sums of +0 or more and a
// bias).  ROUTE_NONE is the key of -inf, 0 that of nothing.
__device__ __forceinline__ uint32_t order_key(float v) {
    const int32_t b = __float_as_int(v);
    return (uint32_t)b ^ ((uint32_t)(b >> 31) | 0x80000000u);
}
constexpr uint32_t ROUTE_NONE = 0x007FFFFFu;

// Two largest of two sorted pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void merge_two(float& a1, float& a2, float b1, float b2) {
    const float lo = fminf(a1, b1);
    a1 = fmaxf(a1, b1);
    a2 = fmaxf(lo, fmaxf(a2, b2));
}

// Positions of this CTA's slots (n of them from slot s0, expert ids at
// `ids`), CTA-size slots at a time; base[e] is the next position of expert e.
// cnt: uint16 [warps][E] in shared memory; ready: it is zero, and `first` is this
// thread's id of the first round.
__device__ __forceinline__ void place_slots(const int32_t* ids, int64_t s0, int n, int E, int* base, uint16_t* cnt,
                                            int32_t* slots, bool ready, int first) {
    const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
    for (int i0 = 0; i0 < n; i0 += nt) {
        const int i = i0 + tid;
        int e = first;
        if (i0 > 0 || !ready) {
            for (int x = tid; x < (nw * E + 1) / 2; x += nt) reinterpret_cast<uint32_t*>(cnt)[x] = 0;
            __syncthreads();
            e = i < n ? ids[i] : -1;
        }
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && rank == 0) cnt[warp * E + e] = (uint16_t)__popc(same);
        __syncthreads();
        for (int x = tid; x < E; x += nt) {                // exclusive prefix over the warps
            int run = 0;
            for (int w0 = 0; w0 < nw; w0 += 8) {           // eight loads in flight
                int c[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) c[w] = w0 + w < nw ? cnt[(w0 + w) * E + x] : 0;
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    if (w0 + w < nw) cnt[(w0 + w) * E + x] = (uint16_t)run;
                    run += c[w];
                }
            }
        }
        __syncthreads();
        if (e >= 0) slots[base[e] + cnt[warp * E + e] + rank] = (int32_t)(s0 + i);
        __syncthreads();
        // advance the bases: the last slot of each expert in the pass knows its end
        if (i0 + nt < n) {
            if (e >= 0) atomicAdd(base + e, 1);            // a count: the order does not matter
            __syncthreads();
        }
    }
}

// Exclusive prefix of v[0..E) in place, v[E] the total, by the whole CTA (in
// rounds of its size); warps: one int a warp, plus one.
__device__ __forceinline__ void exclusive_prefix(int* v, int E, int* warps) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + tid, n = e < E ? v[e] : 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        if (lane == 31) warps[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const int w = lane < nw ? warps[lane] : 0;
            int t = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += up;
            }
            if (lane < nw) warps[lane] = t - w;
            if (lane == 31) warps[nw] = t;
        }
        __syncthreads();
        if (e < E) v[e] = run + warps[warp] + s - n;
        run += warps[nw];
        __syncthreads();
    }
    if (tid == 0) v[E] = run;
    __syncthreads();
}

// The three best keys of a lane and their indices, in the order of the
// selection (larger key, then lower index); REST: of those after (last, at).
struct Best {
    uint32_t k1, k2, k3;
    int i1, i2, i3;
};
template <int V, bool REST>
__device__ __forceinline__ Best three_best(const uint32_t (&key)[V], uint32_t last, int at) {
    Best b{0u, 0u, 0u, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t k = !REST || key[i] < last || (key[i] == last && i > at) ? key[i] : 0u;
        const bool first = k > b.k1, second = k > b.k2, third = k > b.k3;
        b.k3 = second ? b.k2 : third ? k : b.k3;
        b.i3 = second ? b.i2 : third ? i : b.i3;
        b.k2 = first ? b.k1 : second ? k : b.k2;
        b.i2 = first ? b.i1 : second ? i : b.i2;
        b.k1 = first ? k : b.k1;
        b.i1 = first ? i : b.i1;
    }
    return b;
}

// One token: ids and weights, and its experts counted in hist (if any).
// b: the bias of this lane's experts; row_s: E floats of this warp (groups).
template <class T, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t tok, int lane, const float (&b)[V], int* hist,
                                            float* row_s) {
    const unsigned FULL = 0xffffffffu;
    const int e0 = lane * V;
    const T* row = reinterpret_cast<const T*>(a.logits) + tok * a.ld;
    uint32_t key[V];
    float most = 0.f, sum = 1.f;                           // of the softmax
    {
        float l[V], s[V];
        load_row<T, V>(row, a.E, lane, a.vec != 0, l);
        if (a.score == MOE_SOFTMAX) {
#pragma unroll
            for (int i = 0; i < V; ++i) l[i] = available(l[i], b[i]);
            most = l[0];
#pragma unroll
            for (int i = 1; i < V; ++i) most = fmaxf(most, l[i]);
            most = warp_max(most);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = l[i] > -INFINITY ? expf(l[i] - most) : 0.f;
            sum = tree_sum<V>(s);
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = l[i] > -INFINITY ? s[i] / sum + b[i] : -INFINITY;
        } else {
            // (a bias of -inf makes its sum -inf; +inf and the largest f32 have the same sigmoid)
#pragma unroll
            for (int i = 0; i < V; ++i) s[i] = l[i] > -INFINITY ? sigmoid(l[i]) + b[i] : -INFINITY;
        }
        if (a.top_groups < a.groups) {
            float m1 = -INFINITY, m2 = -INFINITY;          // of group lane >> gshift
            const int gs = a.gsize;
            if (a.gwhole) {                                // whole lanes, a power of two
#pragma unroll
                for (int i = 0; i < V; ++i) merge_two(m1, m2, s[i], -INFINITY);
            } else {                                       // its lanes go through its values in shared memory
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + i < a.E) row_s[e0 + i] = s[i];
                __syncwarp();
                const int q = lane >> a.gshift, lanes = 1 << a.gshift;
                if (q < a.groups)
                    for (int i = lane & (lanes - 1); i < gs; i += lanes) merge_two(m1, m2, row_s[q * gs + i], -INFINITY);
                __syncwarp();
            }
            for (int o = 1; o < 1 << a.gshift; o <<= 1) {
                const float q1 = __shfl_xor_sync(FULL, m1, o), q2 = __shfl_xor_sync(FULL, m2, o);
                merge_two(m1, m2, q1, q2);
            }
            const int mine = lane >> a.gshift;
            uint32_t gkey = mine < a.groups ? order_key(m1 + (m2 > -INFINITY ? m2 : 0.f)) : 0u;
            uint32_t in = 0u;                              // groups that take part
            for (int j = 0; j < a.top_groups; ++j) {
                const uint32_t m = __reduce_max_sync(FULL, gkey);
                const int win = (__ffs(__ballot_sync(FULL, gkey == m)) - 1) >> a.gshift;
                in |= 1u << win;
                if (mine == win) gkey = 0u;
            }
            if (a.gwhole) {
                const bool on = (in >> mine) & 1u;
#pragma unroll
                for (int i = 0; i < V; ++i) s[i] = on ? s[i] : -INFINITY;
            } else {
                int grp = e0 / gs, left = (grp + 1) * gs - e0;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (left == 0) {
                        ++grp;
                        left = gs;
                    }
                    --left;
                    if (!((in >> (grp & 31)) & 1u)) s[i] = -INFINITY;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = order_key(s[i]);
    }
    Best top = three_best<V, false>(key, 0u, 0);
    int id = -1, at_hand = 3;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t m = __reduce_max_sync(FULL, top.k1);
        if (m <= ROUTE_NONE) break;                        // none left
        const int win = __ffs(__ballot_sync(FULL, top.k1 == m)) - 1;
        const int e = __shfl_sync(FULL, e0 + top.i1, win);
        if (lane == j) id = e;
        if (lane == win) {
            if (V > 3 && --at_hand == 0) {
                top = three_best<V, true>(key, m, top.i1);
                at_hand = 3;
            } else {
                top = Best{top.k2, top.k3, 0u, top.i2, top.i3, 0};
            }
        }
    }
    // the weights: lane j scores its expert again
    float w = 0.f;
    if (id >= 0) {
        const float l = available(to_f32(row[id]), 0.f);
        w = a.score == MOE_SOFTMAX ? expf(l - most) / sum : sigmoid(l);
    }
    if (a.renorm) w = w / fmaxf(warp_sum(w), ROUTE_TINY);
    if (lane < a.k) {
        a.ids[tok * a.k + lane] = id;
        a.weights[tok * a.k + lane] = w * a.scale;
        if (hist && id >= 0) atomicAdd(hist + id, 1);      // a count: the order does not matter
    }
}

// One CTA a chunk of tokens.  FUSED: the grid is one cluster, which also writes
// the plan.  Shared memory: counts int[E+1]; FUSED: base int[E+1], before
// int[E+1], 33 ints and the warps' counts too.
template <class T, int V, bool FUSED>
__global__ void __launch_bounds__(V <= 8 ? 1024 : 256) moe_route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ int route_smem[];
    int* hist = route_smem;
    const int tid = threadIdx.x, nt = blockDim.x, nw = nt >> 5, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (a.offsets) {
        for (int e = tid; e <= a.E; e += nt) hist[e] = 0;
        __syncthreads();
    }
    pdl_wait();
    float b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        b[i] = a.bias && lane * V + i < a.E ? a.bias[lane * V + i] : 0.f;
        if (!(b[i] > -INFINITY)) b[i] = -INFINITY;         // (a NaN too)
    }
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk;
    const int64_t t1 = t0 + a.chunk < a.T ? t0 + a.chunk : a.T;
    float* row_s = reinterpret_cast<float*>(route_smem + a.off_rows) + warp * a.E;
    for (int64_t t = t0 + warp; t < t1; t += nw) route_token<T, V>(a, t, lane, b, a.offsets ? hist : nullptr, row_s);
    if (!a.offsets) return;
    __syncthreads();
    if (!FUSED) {
        // two experts a word (hist[E] is 0)
        const int words = (a.E + 1) / 2;
        uint32_t* to = reinterpret_cast<uint32_t*>(a.counts) + (int64_t)blockIdx.x * words;
        for (int e = tid; e < words; e += nt) to[e] = (uint32_t)hist[2 * e] | ((uint32_t)hist[2 * e + 1] << 16);
        return;
    }
    int* base = hist + a.E + 1;
    int* before = base + a.E + 1;                          // slots of the CTAs before
    int* warps = before + a.E + 1;
    uint16_t* cnt = reinterpret_cast<uint16_t*>(warps + 34);
    const int rank = (int)blockIdx.x, C = (int)gridDim.x;
    if (C > 1) cluster_sync();                             // every CTA's counts are there
    for (int e = tid; e < a.E; e += nt) {
        int all = 0, ahead = 0;
        for (int c = 0; c < C; ++c) {
            const int v = c == rank ? hist[e] : (int)ld_dsmem_u32(mapa_shared(smem_u32(hist + e), c));
            all += v;
            ahead += c < rank ? v : 0;
        }
        base[e] = all;
        before[e] = ahead;
    }
    if (C > 1) cluster_sync();                             // the counts are read: a CTA may go
    __syncthreads();
    exclusive_prefix(base, a.E, warps);
    const int64_t S = a.T * a.k;
    const int total = base[a.E];
    if (rank == 0)
        for (int e = tid; e <= a.E; e += nt) a.offsets[e] = base[e];
    for (int64_t s = total + rank * nt + tid; s < S; s += C * nt) a.slots[s] = -1;
    __syncthreads();
    for (int e = tid; e < a.E; e += nt) base[e] += before[e];
    __syncthreads();
    // the ids were written by this CTA's own warps (ordered by the barriers above)
    if (t1 > t0) place_slots(a.ids + t0 * a.k, t0 * a.k, (int)((t1 - t0) * a.k), a.E, base, cnt, a.slots, false, -1);
}

// Second kernel of the plan: CTA b places the slots of chunk b.  Shared
// memory: base int[E+2], before int[E+2], 33 ints, the warps' counts.  Every CTA
// sums all chunks' counts (16 bits each, two to a word: 16384 tokens of 256 experts
// are 12 MB out of L2 for all CTAs together).
__global__ void __launch_bounds__(1024) moe_plan_kernel(const int32_t* __restrict__ ids,
                                                        const uint32_t* __restrict__ counts, int chunks, int64_t chunk,
                                                        int64_t T, int E, int k, int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ slots) {
    extern __shared__ int plan_smem[];
    const int words = (E + 1) / 2;
    int* base = plan_smem;                                 // first the totals, then each expert's first position
    int* before = base + 2 * words + 2;                    // slots of earlier chunks
    int* warps = before + 2 * words + 2;
    uint16_t* cnt = reinterpret_cast<uint16_t*>(warps + 34);
    const int tid = threadIdx.x, nt = blockDim.x, b = blockIdx.x;
    pdl_launch_dependents();
    for (int i = tid; i < 2 * words; i += nt) {
        base[i] = 0;
        before[i] = 0;
    }
    for (int i = tid; i < ((nt >> 5) * E + 1) / 2; i += nt) reinterpret_cast<uint32_t*>(cnt)[i] = 0;
    __syncthreads();
    pdl_wait();
    const int64_t t0 = (int64_t)b * chunk, t1 = t0 + chunk < T ? t0 + chunk : T;
    const int n = (int)((t1 - t0) * k);
    const int first = tid < n ? ids[t0 * k + tid] : -1;
    // column sums of the counts, many loads in flight: as many threads to a column as fit
    const int rows = nt / words;
    if (tid < words * rows) {
        const int c0 = tid / words, e = tid - c0 * words;
        const uint32_t* p = counts + e;
        int all0 = 0, all1 = 0, mine0 = 0, mine1 = 0, c = c0;
        auto add = [&](uint32_t v, int at) {
            const int v0 = (int)(v & 0xFFFFu), v1 = (int)(v >> 16);
            all0 += v0;
            all1 += v1;
            mine0 += at < b ? v0 : 0;
            mine1 += at < b ? v1 : 0;
        };
        for (; c + 7 * rows < chunks; c += 8 * rows) {
            uint32_t v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = p[(int64_t)(c + i * rows) * words];
#pragma unroll
            for (int i = 0; i < 8; ++i) add(v[i], c + i * rows);
        }
#pragma unroll 4
        for (; c < chunks; c += rows) add(p[(int64_t)c * words], c);
        atomicAdd(base + 2 * e, all0);                     // counts: the order does not matter
        atomicAdd(base + 2 * e + 1, all1);
        atomicAdd(before + 2 * e, mine0);
        atomicAdd(before + 2 * e + 1, mine1);
    }
    __syncthreads();
    exclusive_prefix(base, E, warps);
    const int64_t S = T * k;
    if (b == 0)
        for (int e = tid; e <= E; e += nt) offsets[e] = base[e];
    for (int64_t s = (int64_t)base[E] + (int64_t)b * nt + tid; s < S; s += (int64_t)gridDim.x * nt) slots[s] = -1;
    __syncthreads();
    for (int i = tid; i < E; i += nt) base[i] += before[i];
    __syncthreads();
    place_slots(ids + t0 * k, t0 * k, n, E, base, cnt, slots, true, first);
}

struct RouteBackArgs {
    const void* logits;
    int64_t ld;
    const float* bias;
    const int32_t* ids;
    const float* dw;
    void* dl;
    int64_t ldd, T;
    int E, k, score, renorm;
    float scale;
    int vec, vecd;
};

// Lane j holds slot j.  Where only the selected logits matter (sigmoid;
// renormalised softmax without a bias, whose selected scores sum to at least
// 1/(2E), so that the common factor of the softmax cancels) they are gathered;
// else the row is read.  A score meets 1 / S before anything else does: g / S alone
// may pass the largest f32, p / S is at most 1.  (A product with the reciprocal: most lanes
// hold no score, and dividing their 0 is slow: 16384x128 sigmoid 5.1 us, now 4.4.)
// A sum below 2^-126 is not what the weights were divided by: they are p times
// a constant there, and so is their gradient.
// The row is written dense, then the selected entries.
template <class T, int V>
__global__ void __launch_bounds__(256) moe_route_backward_kernel(const __grid_constant__ RouteBackArgs a) {
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    const int e0 = lane * V;
    pdl_launch_dependents();
    pdl_wait();
    for (int64_t t = (int64_t)blockIdx.x * nw + (threadIdx.x >> 5); t < a.T; t += (int64_t)gridDim.x * nw) {
        const T* row = reinterpret_cast<const T*>(a.logits) + t * a.ld;
        T* drow = reinterpret_cast<T*>(a.dl) + t * a.ldd;
        const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
        const bool on = id >= 0 && id < a.E;
        const float g = on ? a.dw[t * a.k + lane] * a.scale : 0.f;
        const float l = on ? available(to_f32(row[id]), a.bias ? a.bias[id] : 0.f) : -INFINITY;
        const bool live = l > -INFINITY;
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.f;
        float mine;                                        // gradient of the selected logit
        if (a.score == MOE_SIGMOID) {
            const float p = live ? sigmoid(l) : 0.f, q = live ? sigmoid(-l) : 0.f;   // q = 1 - p without cancellation
            if (a.renorm) {
                // both sums at once, of scores times 2^32, so that g p keeps its bits down to the least p
                const float P = p * 0x1p32f, S = warp_sum(P), gP = warp_sum(g * P);
                const float d = fmaxf(S, ROUTE_TINY * 0x1p32f), one = 1.0f / d;
                mine = P * one * q * (S < d ? g : g - gP * one);
            } else {
                mine = p * q * g;
            }
        } else if (a.renorm && !a.bias) {
            const float m = warp_max(l);
            const float e = live ? expf(l - m) : 0.f;
            const float sum = warp_sum(e);
            const float r = live ? e / sum : 0.f;          // p / S
            mine = r * (g - warp_sum(g * r));
        } else {
            float x[V];
            load_row<T, V>(row, a.E, lane, a.vec != 0, x);
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = available(x[i], a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.f);
                m = fmaxf(m, x[i]);
            }
            m = warp_max(m);
#pragma unroll
            for (int i = 0; i < V; ++i) x[i] = x[i] > -INFINITY ? expf(x[i] - m) : 0.f;
            const float s = tree_sum<V>(x);
            const float p = live ? expf(l - m) / s : 0.f;
            const float S = a.renorm ? warp_sum(p) : 1.f, r = a.renorm ? p * (1.0f / fmaxf(S, ROUTE_TINY)) : p;
            const float dot = warp_sum(g * r);
            // the sum as divisor makes what flows to all experts vanish; a constant one does not
            const bool clamped = a.renorm && S < ROUTE_TINY;
            mine = clamped ? r * g - p * dot : r * (g - dot);
            const float c = (clamped || !a.renorm) && s > 0.f ? -dot / s : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = x[i] * c;
        }
        __syncwarp();                                      // dlogits may be the logits: every lane has read the row
        store_row<T, V>(drow, a.E, lane, a.vecd != 0, out);
        __syncwarp();
        if (on) drow[id] = from_f32<T>(mine);
        __syncwarp();
    }
}

inline bool wide_ok(const void* p, int64_t ld, int E, int V, int size) {
    const int bytes = V * size >= 16 ? 16 : V * size;
    return E % V == 0 && reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * size) % bytes == 0;
}

int experts_a_lane(int E) {
    int V = 1;
    while (32 * V < E) V *= 2;
    return V;
}

template <class F>
cudaError_t raise_smem(F* kernel, size_t smem) {
    if (smem <= 48 * 1024) return cudaSuccess;
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

int sm_count() {
    static std::atomic<int> known[64];                     // never changes: asked once
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 64 && known[dev]) return known[dev];
    int sms = 152;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (dev < 64) known[dev] = sms;
    return sms;
}

template <class T, int V>
cudaError_t launch_route(RouteArgs a, cudaStream_t st) {
    a.vec = wide_ok(a.logits, a.ld, a.E, V, (int)sizeof(T)) ? 1 : 0;
    constexpr int MOST = V <= 8 ? 32 : 8;                  // warps of a CTA
    const size_t head = (size_t)(3 * (a.E + 1) + 34) * 4;
    const bool grouped = a.top_groups < a.groups && !a.gwhole;   // rows pass through shared memory
    // one cluster, a token a warp
    if (a.T <= ROUTE_CLUSTER * MOST) {
        int C = 1;
        while (C < ROUTE_CLUSTER && C * 4 < a.T) C *= 2;   // few tokens a CTA: their instructions bound it
        a.chunk = (a.T + C - 1) / C;
        const int nw = a.chunk < MOST ? (int)a.chunk : MOST;
        a.off_rows = (int)((head + ((size_t)nw * a.E * 2 + 3) / 4 * 4) / 4);
        const size_t smem = (size_t)a.off_rows * 4 + (grouped ? (size_t)nw * a.E * 4 : 0);
        cudaError_t e = raise_smem(moe_route_kernel<T, V, true>, smem);
        if (e == cudaSuccess && C > 8)
            e = cudaFuncSetAttribute(moe_route_kernel<T, V, true>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)C);
        cfg.blockDim = dim3((unsigned)nw * 32);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)C;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = C > 1 ? 2 : 1;
        return cudaLaunchKernelEx(&cfg, moe_route_kernel<T, V, true>, a);
    }
    // a chunk a CTA, at most one CTA of 32 warps (four of 8) on each SM
    int64_t chunks = (a.T + MOST - 1) / MOST;
    const int64_t limit = (int64_t)sm_count() * (MOST == 32 ? 1 : 4), least = (a.T + 65534) / 65535;   // counts of 16 bits
    if (chunks > limit) chunks = limit > least ? limit : least;
    a.chunk = (a.T + chunks - 1) / chunks;
    chunks = (a.T + a.chunk - 1) / a.chunk;
    void* mem = nullptr;
    cudaError_t e = cudaSuccess;
    if (a.offsets) {
        e = scratch_alloc(&mem, (size_t)chunks * ((a.E + 1) / 2) * 4, st);
        if (e != cudaSuccess) return e;
        a.counts = static_cast<uint16_t*>(mem);
    }
    a.off_rows = (int)(head / 4);
    const size_t smem = head + (grouped ? (size_t)MOST * a.E * 4 : 0);
    e = raise_smem(moe_route_kernel<T, V, false>, smem);
    if (e == cudaSuccess)
        e = launch_pdl(moe_route_kernel<T, V, false>, dim3((unsigned)chunks), dim3(MOST * 32), smem, st, a);
    if (e == cudaSuccess && a.offsets) {
        const size_t plan = (size_t)(2 * (a.E + 3) + 34) * 4 + (size_t)32 * a.E * 2;
        e = raise_smem(moe_plan_kernel, plan);
        if (e == cudaSuccess)
            e = launch_pdl(moe_plan_kernel, dim3((unsigned)chunks), dim3(1024), plan, st,
                           static_cast<const int32_t*>(a.ids), reinterpret_cast<const uint32_t*>(a.counts), (int)chunks,
                           a.chunk, a.T, a.E, a.k, a.offsets, a.slots);
    }
    if (mem) {
        const cudaError_t e2 = cudaFreeAsync(mem, st);
        if (e == cudaSuccess) e = e2;
    }
    return e;
}

template <class T, int V>
cudaError_t launch_route_backward(RouteBackArgs a, cudaStream_t st) {
    a.vec = wide_ok(a.logits, a.ld, a.E, V, (int)sizeof(T)) ? 1 : 0;
    a.vecd = wide_ok(a.dl, a.ldd, a.E, V, (int)sizeof(T)) ? 1 : 0;
    int64_t grid = (a.T + 7) / 8;
    if (grid > (int64_t)sm_count() * 8) grid = (int64_t)sm_count() * 8;
    return launch_pdl(moe_route_backward_kernel<T, V>, dim3((unsigned)grid), dim3(256), 0, st, a);
}

template <class T, class A, template <class, int> class L>
cudaError_t by_width(const A& a, int E, cudaStream_t st) {
    switch (experts_a_lane(E)) {
        case 1: return L<T, 1>::go(a, st);
        case 2: return L<T, 2>::go(a, st);
        case 4: return L<T, 4>::go(a, st);
        case 8: return L<T, 8>::go(a, st);
        case 16: return L<T, 16>::go(a, st);
        default: return L<T, 32>::go(a, st);
    }
}
template <class T, int V>
struct Forward {
    static cudaError_t go(const RouteArgs& a, cudaStream_t st) { return launch_route<T, V>(a, st); }
};
template <class T, int V>
struct Backward {
    static cudaError_t go(const RouteBackArgs& a, cudaStream_t st) { return launch_route_backward<T, V>(a, st); }
};
template <class A, template <class, int> class L>
cudaError_t by_type(int dtype, const A& a, int E, cudaStream_t st) {
    if (dtype == TQ2_F32) return by_width<float, A, L>(a, E, st);
    if (dtype == TQ2_F16) return by_width<__half, A, L>(a, E, st);
    return by_width<__nv_bfloat16, A, L>(a, E, st);
}

tq2_status cuda_status(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return TQ2_OK;
    return (tq2_status)set_error(e == cudaErrorMemoryAllocation ? TQ2_ENOMEM : TQ2_ECUDA, "%s: %s", what,
                                 cudaGetErrorString(e));
}

tq2_status check(const char* fn, int64_t ld, int dtype, int64_t T, int E, int k, int score, float scale) {
    if (dtype != TQ2_F32 && dtype != TQ2_F16 && dtype != TQ2_BF16)
        return (tq2_status)set_error(TQ2_EINVAL, "%s: unknown dtype %d", fn, dtype);
    if (score != MOE_SOFTMAX && score != MOE_SIGMOID)
        return (tq2_status)set_error(TQ2_EINVAL, "%s: unknown score %d", fn, score);
    if (!(scale - scale == 0.f)) return (tq2_status)set_error(TQ2_EINVAL, "%s: scale must be finite", fn);
    if (E < 1 || E > 1024 || k < 1 || k > 32 || k > E || T < 0 || T > (1 << 24) || T * k > (1 << 24))
        return (tq2_status)set_error(TQ2_ESHAPE,
                                     "%s: need 1 <= E <= 1024, 1 <= k <= min(E, 32), T*k <= 2^24 (T=%lld E=%d k=%d)",
                                     fn, (long long)T, E, k);
    if (ld < E) return (tq2_status)set_error(TQ2_ESHAPE, "%s: row stride %lld is shorter than E=%d", fn, (long long)ld, E);
    return TQ2_OK;
}

}  // namespace
}  // namespace tq2

using namespace tq2;

extern "C" {

tq2_status moe_route(const void* logits, int64_t ld, int dtype, const float* bias, int64_t T, int E, int k, int score,
                     int groups, int top_groups, int renorm, float scale, int32_t* ids, float* weights,
                     int32_t* offsets, int32_t* slots, void* stream) {
    const tq2_status s = check("moe_route", ld, dtype, T, E, k, score, scale);
    if (s != TQ2_OK) return s;
    if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups)
        return (tq2_status)set_error(TQ2_ESHAPE, "moe_route: bad groups (E=%d groups=%d top_groups=%d)", E, groups,
                                     top_groups);
    if ((offsets == nullptr) != (slots == nullptr) && T > 0)
        return (tq2_status)set_error(TQ2_EINVAL, "moe_route: offsets and slots go together");
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (offsets) return cuda_status(cudaMemsetAsync(offsets, 0, (size_t)(E + 1) * 4, st), "moe_route");
        return TQ2_OK;
    }
    if (!logits || !ids || !weights) return (tq2_status)set_error(TQ2_EINVAL, "moe_route: null pointer");
    if (off_element(logits, element_size(dtype)) || off_element(bias, 4) || off_element(ids, 4) ||
        off_element(weights, 4) || off_element(offsets, 4) || off_element(slots, 4))
        return (tq2_status)set_error(TQ2_EINVAL, "moe_route: pointers must be element-aligned");
    RouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.score = score;
    a.groups = groups;
    a.top_groups = top_groups;
    a.gsize = E / groups;
    const int V = experts_a_lane(E), per = a.gsize / V;
    a.gwhole = per * V == a.gsize && (per & (per - 1)) == 0;
    // else the lanes of a warp are shared out among the groups
    while (a.gwhole ? (2 << a.gshift) <= per : (2 << a.gshift) * groups <= 32) ++a.gshift;
    a.renorm = renorm;
    a.scale = scale;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.slots = slots;
    return cuda_status(by_type<RouteArgs, Forward>(dtype, a, E, st), "moe_route");
}

tq2_status moe_route_backward(const void* logits, int64_t ld, int dtype, const float* bias, const int32_t* ids,
                              const float* dweights, void* dlogits, int64_t ldd, int64_t T, int E, int k, int score,
                              int renorm, float scale, void* stream) {
    const tq2_status s = check("moe_route_backward", ld < ldd ? ld : ldd, dtype, T, E, k, score, scale);
    if (s != TQ2_OK) return s;
    if (T == 0) return TQ2_OK;
    if (!logits || !ids || !dweights || !dlogits)
        return (tq2_status)set_error(TQ2_EINVAL, "moe_route_backward: null pointer");
    if (off_element(logits, element_size(dtype)) || off_element(dlogits, element_size(dtype)) || off_element(bias, 4) ||
        off_element(ids, 4) || off_element(dweights, 4))
        return (tq2_status)set_error(TQ2_EINVAL, "moe_route_backward: pointers must be element-aligned");
    RouteBackArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.bias = bias;
    a.ids = ids;
    a.dw = dweights;
    a.dl = dlogits;
    a.ldd = ldd;
    a.T = T;
    a.E = E;
    a.k = k;
    a.score = score;
    a.renorm = renorm;
    a.scale = scale;
    return cuda_status(by_type<RouteBackArgs, Backward>(dtype, a, E, reinterpret_cast<cudaStream_t>(stream)),
                       "moe_route_backward");
}

}  // extern "C"
