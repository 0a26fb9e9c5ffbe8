// moe_route.cu -- a mixture-of-experts router: scores, groups, top-k,
// renormalised weights, the plan (slots ordered by expert), and the gradient
// of the weights to the logits.
//
// A warp takes a token.  Lane i holds experts i*V .. i*V+V-1 in registers, so
// a row is read once in wide loads, the lowest lane that holds a maximum also
// holds the lowest expert, and the softmax sum's tree over neighbouring
// experts is V-1 additions in the lane and five shuffles.  Selection values
// are compared as order-preserving 32-bit keys: one redux.max and one ballot
// for each of the k experts, and only the winner's lane looks for its next
// best.
//
// The plan is a stable counting sort of the T*k slots.  Up to 32 tokens one
// CTA does all of it.  Beyond, each CTA of the routing kernel leaves its
// chunk's counts, and a second kernel (its launch overlaps the first)
// turns them into each chunk's first positions and writes the slots: within
// a chunk, warps count their 32 slots by match.any and a prefix over the
// warps orders them, so there is no atomic whose order could matter.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/tq2.h"
#include "ptx.cuh"
#include "tq2_internal.h"

namespace tq2 {

namespace {

constexpr float ROUTE_TINY = 1.17549435e-38f;      // 2^-126
constexpr float ROUTE_MOST = 3.402823466e+38f;     // largest f32
constexpr int ROUTE_FUSED = 32;                    // tokens that one CTA plans in the routing kernel

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
    int32_t* counts;                               // [chunks][E], two-kernel plan
    int64_t chunk;                                 // tokens of a CTA
    int vec;                                       // rows can be read in wide loads
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
        }
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = e0 < E ? to_f32(raw[i]) : -INFINITY;
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
__device__ __forceinline__ float sigmoid(float l) { return 1.0f / (1.0f + expf(-l)); }

// Larger value, larger key; 0 is below every number's key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);          // -0 and 0 compare equal
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Two largest of two sorted pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void merge_two(float& a1, float& a2, float b1, float b2) {
    const float lo = fminf(a1, b1);
    a1 = fmaxf(a1, b1);
    a2 = fmaxf(lo, fmaxf(a2, b2));
}

// Positions of this CTA's slots (n of them from slot s0, expert ids at
// `ids`), CTA-size slots at a time; base[e] is the next position of expert e.
// cnt: uint16 [warps][E] in shared memory.
__device__ __forceinline__ void place_slots(const int32_t* ids, int64_t s0, int n, int E, int* base, uint16_t* cnt,
                                            int32_t* slots) {
    const int tid = threadIdx.x, nt = blockDim.x, warp = tid >> 5, lane = tid & 31, nw = nt >> 5;
    for (int i0 = 0; i0 < n; i0 += nt) {
        for (int i = tid; i < nw * E; i += nt) cnt[i] = 0;
        __syncthreads();
        const int i = i0 + tid;
        const int e = i < n ? ids[i] : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        if (e >= 0 && rank == 0) cnt[warp * E + e] = (uint16_t)__popc(same);
        __syncthreads();
        for (int x = tid; x < E; x += nt) {                // exclusive prefix over the warps
            int run = 0;
            for (int w = 0; w < nw; ++w) {
                const int c = cnt[w * E + x];
                cnt[w * E + x] = (uint16_t)run;
                run += c;
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

// Exclusive prefix of v[0..E) in place by the first warp; returns nothing, v[E] the total.
__device__ __forceinline__ void exclusive_prefix(int* v, int E, int lane) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int e = e0 + lane, n = e < E ? v[e] : 0;
        int s = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += up;
        }
        if (e < E) v[e] = run + s - n;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) v[E] = run;
}

template <class T, int V>
__device__ __forceinline__ void route_token(const RouteArgs& a, int64_t tok, int lane, int* hist) {
    const unsigned FULL = 0xffffffffu;
    const int e0 = lane * V;
    float l[V], p[V];
    load_row<T, V>(reinterpret_cast<const T*>(a.logits) + tok * a.ld, a.E, lane, a.vec != 0, l);
    float b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = available(l[i], b[i]);
    if (a.score == MOE_SOFTMAX) {
        float m = l[0];
#pragma unroll
        for (int i = 1; i < V; ++i) m = fmaxf(m, l[i]);
        m = warp_max(m);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = l[i] > -INFINITY ? expf(l[i] - m) : 0.f;
        const float s = tree_sum<V>(p);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = l[i] > -INFINITY ? p[i] / s : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = l[i] > -INFINITY ? sigmoid(l[i]) : 0.f;
    }
    uint32_t key[V];
    {
        float s[V];
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] = l[i] > -INFINITY ? (a.bias ? p[i] + b[i] : p[i]) : -INFINITY;
        uint32_t in = FULL;                                // groups that take part
        const int gs = a.E / a.groups;
        const bool grouped = a.top_groups < a.groups;
        if (grouped) {
            float value = -INFINITY;                       // of group `lane`
            const int per = gs / V;                        // lanes of a group, where it is whole lanes
            if (per * V == gs && (per & (per - 1)) == 0) {
                float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                for (int i = 0; i < V; ++i) merge_two(m1, m2, s[i], -INFINITY);
                for (int o = 1; o < per; o <<= 1) {
                    const float q1 = __shfl_xor_sync(FULL, m1, o), q2 = __shfl_xor_sync(FULL, m2, o);
                    merge_two(m1, m2, q1, q2);
                }
                const float two = m1 + (m2 > -INFINITY ? m2 : 0.f);
                value = __shfl_sync(FULL, two, (lane * per) & 31);
                if (lane >= a.groups) value = -INFINITY;
            } else {
                for (int q = 0; q < a.groups; ++q) {
                    float m1 = -INFINITY, m2 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        if (e0 + i >= q * gs && e0 + i < (q + 1) * gs) merge_two(m1, m2, s[i], -INFINITY);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float q1 = __shfl_xor_sync(FULL, m1, o), q2 = __shfl_xor_sync(FULL, m2, o);
                        merge_two(m1, m2, q1, q2);
                    }
                    if (lane == q) value = m1 + (m2 > -INFINITY ? m2 : 0.f);
                }
            }
            int before = 0;                                // groups ahead of this one
            for (int q = 0; q < a.groups; ++q) {
                const float o = __shfl_sync(FULL, value, q);
                before += (o > value || (o == value && q < lane)) ? 1 : 0;
            }
            in = __ballot_sync(FULL, lane < a.groups && before < a.top_groups);
        }
        int grp = grouped ? e0 / gs : 0, left = grouped ? (grp + 1) * gs - e0 : V;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (left == 0) {
                ++grp;
                left = gs;
            }
            --left;
            key[i] = s[i] > -INFINITY && ((in >> (grp & 31)) & 1u) ? order_key(s[i]) : 0u;
        }
    }
    uint32_t best = 0;
    int bi = 0;
    float bp = 0.f;
    auto look = [&]() {
        best = 0;
        bi = 0;
        bp = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > best) {
                best = key[i];
                bi = i;
                bp = p[i];
            }
    };
    look();
    int id = -1;
    float w = 0.f;
    for (int j = 0; j < a.k; ++j) {
        const uint32_t m = __reduce_max_sync(FULL, best);
        if (m == 0u) break;                                // none left
        const int win = __ffs(__ballot_sync(FULL, best == m)) - 1;
        const int e = __shfl_sync(FULL, e0 + bi, win);
        const float q = __shfl_sync(FULL, bp, win);
        if (lane == j) {
            id = e;
            w = q;
        }
        if (lane == win) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == bi) key[i] = 0u;
            look();
        }
    }
    if (a.renorm) w = w / fmaxf(warp_sum(w), ROUTE_TINY);
    if (lane < a.k) {
        a.ids[tok * a.k + lane] = id;
        a.weights[tok * a.k + lane] = w * a.scale;
        if (hist && id >= 0) atomicAdd(hist + id, 1);      // a count: the order does not matter
    }
}

// One CTA a chunk of tokens.  FUSED: one CTA for all of them, which also
// writes the plan.  Shared memory: counts int[E+1]; FUSED: the ids of the
// chunk and the warps' counts too.
template <class T, int V, bool FUSED>
__global__ void __launch_bounds__(V <= 8 ? 1024 : 256) moe_route_kernel(const __grid_constant__ RouteArgs a) {
    extern __shared__ int route_smem[];
    int* hist = route_smem;
    const int tid = threadIdx.x, nw = blockDim.x >> 5, warp = tid >> 5, lane = tid & 31;
    pdl_launch_dependents();
    if (a.offsets) {
        for (int e = tid; e <= a.E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
    }
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * a.chunk;
    const int64_t t1 = t0 + a.chunk < a.T ? t0 + a.chunk : a.T;
    for (int64_t t = t0 + warp; t < t1; t += nw) route_token<T, V>(a, t, lane, a.offsets ? hist : nullptr);
    if (!a.offsets) return;
    __syncthreads();
    if (!FUSED) {
        for (int e = tid; e < a.E; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
        return;
    }
    if (warp == 0) exclusive_prefix(hist, a.E, lane);
    __syncthreads();
    const int S = (int)(a.T * a.k), total = hist[a.E];
    for (int e = tid; e <= a.E; e += blockDim.x) a.offsets[e] = hist[e];
    for (int s = total + tid; s < S; s += blockDim.x) a.slots[s] = -1;
    // the ids were written by this CTA's own warps (ordered by the barrier above)
    place_slots(a.ids, 0, S, a.E, hist, reinterpret_cast<uint16_t*>(hist + a.E + 1 + (a.E + 1) % 2), a.slots);
}

// Second kernel of the plan: CTA b places the slots of chunk b.  Shared
// memory: base int[E+1], part int[2*E], the warps' counts.
__global__ void __launch_bounds__(1024) moe_plan_kernel(const int32_t* __restrict__ ids,
                                                        const int32_t* __restrict__ counts, int chunks, int64_t chunk,
                                                        int64_t T, int E, int k, int32_t* __restrict__ offsets,
                                                        int32_t* __restrict__ slots) {
    extern __shared__ int plan_smem[];
    int* base = plan_smem;                                 // first the totals, then each expert's first position
    int* before = base + E + 1;                            // slots of earlier chunks
    uint16_t* cnt = reinterpret_cast<uint16_t*>(before + E + (E + 1 + E) % 2);
    const int tid = threadIdx.x, nt = blockDim.x, b = blockIdx.x;
    pdl_launch_dependents();
    for (int i = tid; i < E; i += nt) {
        base[i] = 0;
        before[i] = 0;
    }
    __syncthreads();
    pdl_wait();
    // column sums of the counts: as many threads to a column as fit
    const int cols = E < nt ? E : nt, rows = nt / cols;
    if (tid < cols * rows)
        for (int e = tid % cols; e < E; e += cols) {
            int all = 0, mine = 0;
#pragma unroll 8
            for (int c = tid / cols; c < chunks; c += rows) {
                const int v = counts[(int64_t)c * E + e];
                all += v;
                mine += c < b ? v : 0;
            }
            atomicAdd(base + e, all);                      // counts: the order does not matter
            atomicAdd(before + e, mine);
        }
    __syncthreads();
    if (tid < 32) exclusive_prefix(base, E, tid);
    __syncthreads();
    const int64_t S = T * k;
    if (b == 0)
        for (int e = tid; e <= E; e += nt) offsets[e] = base[e];
    for (int64_t s = (int64_t)base[E] + (int64_t)b * nt + tid; s < S; s += (int64_t)gridDim.x * nt) slots[s] = -1;
    __syncthreads();
    for (int i = tid; i < E; i += nt) base[i] += before[i];
    __syncthreads();
    const int64_t t0 = (int64_t)b * chunk, t1 = t0 + chunk < T ? t0 + chunk : T;
    place_slots(ids + t0 * k, t0 * k, (int)((t1 - t0) * k), E, base, cnt, slots);
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
// else the row is read.  The row is written dense, then the selected entries.
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
        float g = on ? a.dw[t * a.k + lane] * a.scale : 0.f;
        const float l = on ? available(to_f32(row[id]), a.bias ? a.bias[id] : 0.f) : -INFINITY;
        const bool live = l > -INFINITY;
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.f;
        float mine;                                        // gradient of the selected logit
        if (a.score == MOE_SIGMOID) {
            const float p = live ? sigmoid(l) : 0.f, q = live ? sigmoid(-l) : 0.f;   // q = 1 - p without cancellation
            if (a.renorm) {
                const float S = fmaxf(warp_sum(p), ROUTE_TINY);
                g = (g - warp_sum(g * p) / S) / S;
            }
            mine = p * q * g;
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
            float dot = 0.f;
            if (a.renorm) {
                const float S = fmaxf(warp_sum(p), ROUTE_TINY);
                g = (g - warp_sum(g * p) / S) / S;
            } else {
                dot = warp_sum(g * p);
            }
            mine = p * (g - dot);
            const float c = s > 0.f ? -dot / s : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) out[i] = x[i] * c;
        }
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

template <class T, int V>
cudaError_t launch_route(RouteArgs a, cudaStream_t st) {
    a.vec = wide_ok(a.logits, a.ld, a.E, V, (int)sizeof(T)) ? 1 : 0;
    constexpr int MOST = V <= 8 ? 32 : 8;                  // warps of a CTA
    const size_t head = (size_t)(a.E + 1 + (a.E + 1) % 2) * 4;
    if (a.T <= ROUTE_FUSED) {
        const int nw = a.T < MOST ? (int)a.T : MOST;
        a.chunk = a.T;
        const size_t smem = head + (size_t)nw * a.E * 2;
        if (smem > 48 * 1024) {
            cudaError_t e = cudaFuncSetAttribute(moe_route_kernel<T, V, true>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) return e;
        }
        return launch_pdl(moe_route_kernel<T, V, true>, dim3(1), dim3(nw * 32), smem, st, a);
    }
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // a chunk a CTA, at most one CTA of 32 warps (four of 8) on each SM
    int64_t chunks = (a.T + MOST - 1) / MOST;
    const int64_t limit = (int64_t)sms * (MOST == 32 ? 1 : 4);
    if (chunks > limit) chunks = limit;
    a.chunk = (a.T + chunks - 1) / chunks;
    chunks = (a.T + a.chunk - 1) / a.chunk;
    void* mem = nullptr;
    cudaError_t e = cudaSuccess;
    if (a.offsets) {
        e = scratch_alloc(&mem, (size_t)chunks * a.E * 4, st);
        if (e != cudaSuccess) return e;
        a.counts = static_cast<int32_t*>(mem);
    }
    e = launch_pdl(moe_route_kernel<T, V, false>, dim3((unsigned)chunks), dim3(MOST * 32), head, st, a);
    if (e == cudaSuccess && a.offsets) {
        const size_t smem = (size_t)(2 * a.E + 2) * 4 + (size_t)32 * a.E * 2;
        if (smem > 48 * 1024)
            e = cudaFuncSetAttribute(moe_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
            e = launch_pdl(moe_plan_kernel, dim3((unsigned)chunks), dim3(1024), smem, st,
                           static_cast<const int32_t*>(a.ids), static_cast<const int32_t*>(a.counts), (int)chunks,
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
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    int64_t grid = (a.T + 7) / 8;
    if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
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
    if (E < 1 || E > 1024 || k < 1 || k > 32 || k > E || T < 0 || T * k > (1 << 24) || T > (1 << 24))
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
