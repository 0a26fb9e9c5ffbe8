// kv8_stream.cu -- attention of few rows over the 8-bit cache: decoded and
// drafted tokens.
//
// Mathematics, per row r (a query token and one of its heads) and token t, with the
// scales ks and vs of the token's block:
//     w_t = scale log2(e) ks (q_r . c_t) + x_t,   x_t the exponent of vs = 2^x_t f_t
//     out = 2^(m - n) sum_t 2^(w_t - m) f_t c'_t / l,  l = sum_t 2^(w_t - m) 2^(m - n - x_t)
// so that what is rounded to f16 is the whole weight of a value code c': a block of large
// values takes no bits from others that it does not outweigh.  m and n are running references
// that follow the largest w and w - x in steps, so that few tokens rescale the sums.
// The codes are whole numbers, exact in f16; f16 and bf16 queries, scaled by a power of
// two a row, are exact as well, f32 ones are two f16 parts (and so are their
// weights), of which an MMA takes both as rows r and r + 8.  Sums are f32.
//
// Bound: the bytes of the codes (64 tokens of up to 8192, 8 heads of 128, G = 4, bf16: 103 us, 5.1 TB/s or 76 % of the
// measured copy; 400 warp instructions for 16 tokens' 4 KB keep the issue slots 45 % busy).  One sequence of
// 131072 tokens, 4 heads: 37.6 us, 32 of them here and the rest in the join of 76 pieces a head.  The fence before a stage
// goes back costs 1 to 2 %.
// A CTA walks chunks of 64 tokens; all chunks of all sequences and heads are cut over the CTAs by what they cost, so a
// ragged batch or one long sequence fills the GPU alike.  What a cut divides is joined by a second
// kernel in the order of the tokens.  TMA brings the chunks into a ring (keys and values of
// a chunk are swizzled rows, so that fragments are read without conflicts), four warps take 16
// tokens of each; two CTAs an SM with four chunks ahead (104 us and 53 when both were
// measured; three with three, and 128 registers, 107 and 65, the first 149 where calls overlap).
// The codes go from bytes into f16 pairs by a permutation under the exponent of 1024 and one subtraction.
#include <cfloat>
#include <type_traits>

#include "kv8_join.cuh"
#include "q4.cuh"

namespace tq2 {
namespace {

constexpr int CT = 64;          // tokens of a chunk
constexpr int WARPS = 4;        // that compute; one more feeds them
constexpr int THREADS = WARPS * 32 + 32;
constexpr int STAGES = 4;
constexpr int CTAS = 2;         // a SM
// The running reference m of a row: HEAD below the largest weight when it was set (so that f16 keeps
// weights down to 2^-30 of it), set anew where a weight passes RAISE above it (2^15 is in f16's range).
constexpr float HEAD = 6.f, RAISE = 14.f;
// The cut counts a tile of rows as its chunks and so many more, which is about what queries and the closing sums
// cost.  A cut through those is one at their start.  (1, 2, 3, 4: 64 sequences of up to 8192 tokens, 8 heads, G = 4, 110,
// 105, 103, 103.5 us; 256 of 1024 91, 82, 78, 78; one of 131072 alike.)
constexpr int EXTRA = 3;
constexpr int LEAST = EXTRA + 1;                             // units of a CTA: no two cuts through the same EXTRA

template <int D>
struct __align__(1024) Shared {
    uint8_t k[STAGES][CT * D];
    uint8_t v[STAGES][CT * D];
    uint4 q[D / 16][32];        // queries as MMA operands, by k step and lane
    float acc[WARPS][16 * (D / 2 + 4)];
    float m[WARPS][16], l[WARPS][16], n[WARPS][16];
    float qa[16];               // what undoes a row's power of two
    float2 scales[STAGES][4];   // of keys and of values, by piece; values' -1: nothing there
    uint64_t full[STAGES], empty[STAGES];
    long long sums[WARPS + 1], seq_start;
    int seq;
    volatile int abort;
};

struct Walk {
    // a CTA's chunks [pos, end) of the whole list; the current sequence's begin at `base`
    long long pos, end, base;
    int s;
    Kv8Seq q;
    int tiles, first, count;    // row tiles of a head, first chunk, chunks of a tile
};

template <int RM>
__device__ __forceinline__ long long open_seq(const Kv8Attention& a, int s, Walk& w) {
    w.s = s;
    w.q = kv8_seq(a.c, s);
    const int rows = w.q.n * a.G;
    w.tiles = rows > a.few ? 0 : (rows + RM - 1) / RM;
    const int from = a.window ? max(w.q.len - w.q.n - a.window + 1, 0) : 0;
    w.first = from / CT;
    w.count = max((w.q.len + CT - 1) / CT - w.first, 1);
    return (long long)w.tiles * a.c.H * (w.count + EXTRA);
}

// Barrier of the computing warps; the second tells all of them whether any gave up.
__device__ __forceinline__ void named_sync() { asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory"); }
__device__ __forceinline__ bool named_sync_or(bool any) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)any), "n"(WARPS * 32)
        : "memory");
    return r != 0;
}

// SPLIT: tiles of 8 rows, an MMA's rows r + 8 hold second parts: of f32 queries and weights, and of f16 results' weights
// where there are no more than 8 rows (with more, those take MMAs of their own: TWO).
template <class T, int D, bool SPLIT>
__global__ void __launch_bounds__(THREADS, CTAS)
kv8_stream_kernel(const __grid_constant__ Kv8Attention a, float* parts, Kv8Joint* joints) {
    // weights of f16 outputs in two parts too: one part's rounding is as large as the output's own
    constexpr bool TWO = !SPLIT && std::is_same<T, __half>::value;
    constexpr int RM = SPLIT ? 8 : 16;
    constexpr int NT = D / 8;                                // column tiles of the output
    extern __shared__ __align__(1024) uint8_t raw[];
    Shared<D>& sm = *reinterpret_cast<Shared<D>*>(raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&sm.full[i], 33);
            mbar_init(&sm.empty[i], WARPS);
        }
        sm.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.map);
    }
    pdl_launch_dependents();
    pdl_wait();

    // the whole list's length, and where this CTA's share begins
    const int S = a.c.seqs, per = (S + THREADS - 1) / THREADS;
    Walk w;
    long long mine = 0;
    for (int s = tid * per; s < min((tid + 1) * per, S); ++s) mine += open_seq<RM>(a, s, w);
    long long before = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, before, d);
        if (lane >= d) before += u;
    }
    if (lane == 31) sm.sums[warp] = before;
    before -= mine;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int i = 0; i <= WARPS; ++i) {
        if (i < warp) before += sm.sums[i];
        total += sm.sums[i];
    }
    const Kv8Cut cut(total, gridDim.x, LEAST);
    const int cta = blockIdx.x;
    if (cta >= cut.ctas) {
        if (tid == 0) joints[cta].pieces = 0;
        return;
    }
    w.pos = cut.begin(cta);
    w.end = cut.begin(cta + 1);
    if (before <= w.pos && w.pos < before + mine) {
        for (int s = tid * per;; ++s) {
            const long long len = open_seq<RM>(a, s, w);
            if (w.pos < before + len) {
                sm.seq = s;
                sm.seq_start = before;
                break;
            }
            before += len;
        }
    }
    __syncthreads();
    w.base = sm.seq_start;
    long long span = open_seq<RM>(a, sm.seq, w);
    {
        const int at = (int)((w.pos - w.base) % (w.count + EXTRA));
        if (at <= EXTRA) w.pos -= at;
    }
    const int logB = a.c.logB;
    const int rows_piece = min(1 << logB, CT), pieces = CT / rows_piece;

    if (warp == WARPS) {
        // ------------------------------------------------------- producer
        int stage = 0, phase = 0;
        bool issued = false;                                 // all stages have been
        fence_proxy_async_shared();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        while (w.pos < w.end) {
            while (w.pos >= w.base + span) {
                w.base += span;
                span = open_seq<RM>(a, w.s + 1, w);
            }
            const long long in = w.pos - w.base;
            const int item = (int)(in / (w.count + EXTRA)), at = (int)(in % (w.count + EXTRA));
            const int head = item / w.tiles;
            const int take = (int)min((long long)(w.count + EXTRA - at), w.end - w.pos);
            const int run = take - (at ? 0 : EXTRA), ch = at ? at - EXTRA : 0;
            const int from = a.window ? max(w.q.len - w.q.n - a.window + 1, 0) : 0;
            for (int i = 0; i < run; ++i) {
                if (!kv8_wait(&sm.empty[stage], phase ^ 1, &sm.abort, false)) {
                    // copies in flight end before the shared memory goes
                    for (int u = 0; u < STAGES; ++u) {
                        if (u < stage || issued) mbar_wait(&sm.full[u], u < stage ? phase : phase ^ 1);
                    }
                    return;
                }
                const int token = (w.first + ch + i) * CT + lane * rows_piece;
                int block = -1;
                if (lane < pieces) {
                    if (token < w.q.len && token + rows_piece > from) block = kv8_block(a.c, w.s, token);
                    if (block < 0) sm.scales[stage][lane] = make_float2(0.f, -1.f);
                }
                const uint32_t here = __ballot_sync(0xffffffffu, block >= 0);
                __syncwarp();                                // the ordinary stores are lane 0's to release
                if (lane == 0)
                    mbar_arrive_expect_tx(&sm.full[stage], __popc(here) * 2u * (uint32_t)(rows_piece * D));
                if (block >= 0) {
                    const int inside = token & ((1 << logB) - 1);
                    const int64_t kr = kv8_row(a.c, block, 0, head) + inside, vr = kv8_row(a.c, block, 1, head) + inside;
                    tma_load_2d(sm.k[stage] + lane * rows_piece * D, &a.map, &sm.full[stage], 0, (int)kr);
                    tma_load_2d(sm.v[stage] + lane * rows_piece * D, &a.map, &sm.full[stage], 0, (int)vr);
                    const float* sc = a.c.scales + (int64_t)block * 2 * a.c.H + head;
                    cp_async4(&sm.scales[stage][lane].x, sc);
                    cp_async4(&sm.scales[stage][lane].y, sc + a.c.H);
                }
                cp_async_arrive(&sm.full[stage]);
                if (++stage == STAGES) stage = 0, phase ^= 1, issued = true;
            }
            w.pos += take;
        }
        return;
    }

    // ----------------------------------------------------------- consumers
    const int g = lane >> 2, t4 = lane & 3;
    int stage = 0, phase = 0;
    Kv8Joint joint{0, 0, 0, 0};
    bool ok = true;
    while (w.pos < w.end) {
        while (w.pos >= w.base + span) {
            w.base += span;
            span = open_seq<RM>(a, w.s + 1, w);
        }
        const long long in = w.pos - w.base;
        const int item = (int)(in / (w.count + EXTRA)), at = (int)(in % (w.count + EXTRA));
        const int head = item / w.tiles, tile = item % w.tiles;
        const int take = (int)min((long long)(w.count + EXTRA - at), w.end - w.pos);
        const int run = take - (at ? 0 : EXTRA), ch = at ? at - EXTRA : 0;
        if (run <= 0) break;                                 // the next CTA begins with these rows
        const int rows = min(w.q.n * a.G - tile * RM, RM);

        // The tile's queries as MMA operands: k step 4j+i of lane 4g+t takes elements D/4 t + 16j + 4i + {0,1}, {2,3}
        // of rows g and g + 8 (SPLIT: of row g, first parts and second).  Eight lanes read a row.
        {
            constexpr int EL = D / 8;
            const int r = warp * (RM / WARPS) + (lane >> 3);
            const bool mine = lane >> 3 < RM / WARPS, live = mine && r < rows;
            const int rr = tile * RM + (live ? r : 0), j = rr / a.G;
            const int d0 = (lane & 7) * EL;
            const T* p = static_cast<const T*>(a.q) + (int64_t)(w.q.q0 + j) * a.qt + (int64_t)(head * a.G + rr % a.G) * a.qh + d0;
            float x[EL], most = 0.f;
            if (a.qvec) {
                constexpr int N = 16 / (int)sizeof(T);
#pragma unroll
                for (int e = 0; e < EL; e += N) {
                    const uint4 u = *reinterpret_cast<const uint4*>(p + e);
#pragma unroll
                    for (int k = 0; k < N; ++k) x[e + k] = kv8_wide(reinterpret_cast<const T*>(&u)[k]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < EL; ++e) x[e] = kv8_wide(p[e]);
            }
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                x[e] = live ? x[e] : 0.f;
                most = fmaxf(most, fabsf(x[e]));
            }
#pragma unroll
            for (int d = 1; d < 8; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
            const int e = kv8_power(most);
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
            if (mine) {
                // (a row that has an Inf is none of numbers: its scores might all be -Inf, as if it saw no token)
                if ((lane & 7) == 0)
                    sm.qa[r] = most <= FLT_MAX ? a.scale * __uint_as_float((uint32_t)(127 - e) << 23) : __int_as_float(0x7fffffff);
                const int half = SPLIT ? 0 : r >> 3, to = (r & 7) * 4 + d0 / (D / 4), in_quarter = d0 % (D / 4);
#pragma unroll
                for (int i = 0; i < EL; i += 2) {
                    const float u0 = x[i] * up, u1 = x[i + 1] * up;
                    const uint32_t h = pack_half2(u0, u1);
                    uint32_t* dst = reinterpret_cast<uint32_t*>(&sm.q[(in_quarter + i) / 4][to]) + (i % 4 / 2) * 2;
                    dst[half] = h;
                    if (SPLIT) dst[1] = rest_half2(u0, u1, h);
                }
            }
        }
        named_sync();
        float qa[2];
        int hi[2], lo[2];
        constexpr int HALVES = SPLIT ? 1 : 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = g + 8 * (SPLIT ? 0 : half);
            const int pos = w.q.len - w.q.n + (tile * RM + (r < rows ? r : 0)) / a.G;
            qa[half] = sm.qa[r];
            hi[half] = a.causal ? min(w.q.len, pos + 1) : w.q.len;
            lo[half] = a.window ? max(pos - a.window + 1, 0) : 0;
        }
        // tokens [safe_lo, safe_hi) are seen by all rows of the tile
        const int j0 = tile * RM / a.G, j1 = (tile * RM + rows - 1) / a.G;
        const int p0 = w.q.len - w.q.n + j0, p1 = w.q.len - w.q.n + j1;
        const int safe_hi = a.causal ? min(w.q.len, p0 + 1) : w.q.len;
        const int safe_lo = a.window ? max(p1 - a.window + 1, 0) : 0;
        const int any_hi = a.causal ? min(w.q.len, p1 + 1) : w.q.len;
        const int any_lo = a.window ? max(p0 - a.window + 1, 0) : 0;

        float acc[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        const float NONE = kv8_none();
        float m[2] = {NONE, NONE}, l[2] = {0.f, 0.f}, n[2] = {NONE, NONE};
        float ratio[2] = {0.f, 0.f};                         // 2^(m - n)

        for (int i = 0; i < run && ok; ++i) {
            ok = kv8_wait(&sm.full[stage], phase, &sm.abort, false);
            if (!ok) break;
            const int token = (w.first + ch + i) * CT + warp * 16;
            const float2 sc = sm.scales[stage][(warp * 16) / rows_piece];
            if (!(sc.y < 0.f) && token < any_hi && token + 16 > any_lo) {
                // ---- scores of 16 tokens
                float s[2][4] = {};
#pragma unroll
                for (int c = 0; c < D / 64; ++c) {
                    uint4 kw[2];
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        const int row = warp * 16 + n * 8 + g;
                        const int col = D == 128 ? (2 * t4 + c) ^ (row & 7) : t4 ^ ((row >> 1) & 3);
                        kw[n] = *reinterpret_cast<const uint4*>(sm.k[stage] + row * D + col * 16);
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const uint4 u = sm.q[4 * c + x][lane];
                        const uint32_t qf[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const uint32_t e = reinterpret_cast<const uint32_t*>(&kw[n])[x];
                            mma_16816_pure(s[n], qf, kv8_pair<0>(e), kv8_pair<2>(e));
                        }
                    }
                }
                // ---- weights
                const bool number = sc.y <= FLT_MAX;         // (values that are none leave NaN in the sums of values alone)
                const uint32_t vb = __float_as_uint(number ? fmaxf(sc.y, 0x1p-103f) : 1.f);
                const int ex = (int)(vb >> 23) - 127;
                const float down = __uint_as_float(max((uint32_t)(127 - ex) << 23, 0x400000u));   // (2^-127 is a subnormal)
                const float frac = number ? sc.y * down : __int_as_float(0x7fffffff);
                const float ks = sc.x <= FLT_MAX ? sc.x : __int_as_float(0x7fffffff);
                const float a0 = ks * qa[0], a1 = ks * qa[1], fex = (float)ex;
                float e0[4], e1[4];                          // rows g and g + 8 (SPLIT: e0 alone)
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        e0[2 * n + x] = fmaf(SPLIT ? s[n][x] + s[n][2 + x] : s[n][x], a0, fex);
                        if (!SPLIT) e1[2 * n + x] = fmaf(s[n][2 + x], a1, fex);
                    }
                const bool inside = token >= safe_lo && token + 16 <= safe_hi;
                if (!inside) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const int t = token + (x >> 1) * 8 + 2 * t4 + (x & 1);
                        if (t < lo[0] || t >= hi[0]) e0[x] = NONE;
                        if (!SPLIT && (t < lo[1] || t >= hi[1])) e1[x] = NONE;
                    }
                }
                float t0 = fmaxf(fmaxf(e0[0], e0[1]), fmaxf(e0[2], e0[3]));
                float t1 = SPLIT ? NONE : fmaxf(fmaxf(e1[0], e1[1]), fmaxf(e1[2], e1[3]));
                float unit[2] = {ratio[0] * down, ratio[1] * down};          // of a weight in l
                if (__any_sync(0xffffffffu, t0 > m[0] + RAISE || t1 > m[1] + RAISE || fmaxf(unit[0], unit[1]) > KV8_FAR)) {
#pragma unroll
                    for (int half = 0; half < HALVES; ++half) {
                        const auto top_of_row = [](float t) {             // the same in a row's four lanes
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                            return fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                        };
                        const auto follow = [&](float to) {
                            if (to > n[half]) l[half] *= exp2_fast(n[half] - to), n[half] = to;
                        };
                        const float t = top_of_row(half ? t1 : t0);
                        if (t > m[half] + RAISE) {
                            const float f = exp2_fast(m[half] - (t - HEAD));
                            m[half] = t - HEAD;
                            follow(m[half] - fex);
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                acc[c][2 * half] *= f;
                                acc[c][2 * half + 1] *= f;
                                if (SPLIT) {
                                    acc[c][2] *= f;
                                    acc[c][3] *= f;
                                }
                            }
                        }
                        unit[half] = m[half] == NONE ? 0.f : exp2_fast(m[half] - n[half]) * down;
                        if (__any_sync(0xffffffffu, unit[half] > KV8_FAR)) {
                            float z[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const float* u = s[x >> 1];
                                z[x] = SPLIT ? (u[x & 1] + u[2 + (x & 1)]) * a0 : u[2 * half + (x & 1)] * (half ? a1 : a0);
                                if (!inside && (half ? e1 : e0)[x] == NONE) z[x] = NONE;
                            }
                            const float most = top_of_row(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
                            if (most > n[half] + RAISE) follow(most - HEAD);
                            const float ref = n[half] == NONE ? 0.f : n[half];
#pragma unroll
                            for (int x = 0; x < 4; ++x) l[half] += exp2_fast(z[x] - ref);
                            unit[half] = 0.f;
                        }
                        ratio[half] = m[half] == NONE ? 0.f : exp2_fast(m[half] - n[half]);
                    }
                }
                uint32_t pf[4], pl[4];
                {
                    const float m0 = m[0] == NONE ? 0.f : m[0];
                    float sum = 0.f;                         // (without a reference 0 or NaN)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const bool dead = !inside && e0[x] == NONE;
                        const float e = exp2_fast(e0[x] - m0);
                        sum += e;
                        e0[x] = dead ? 0.f : e * frac;
                    }
                    l[0] = fmaf(sum, unit[0], l[0]);
                    pf[0] = pack_half2(e0[0], e0[1]);
                    pf[2] = pack_half2(e0[2], e0[3]);
                    if (SPLIT) {
                        pf[1] = rest_half2(e0[0], e0[1], pf[0]);
                        pf[3] = rest_half2(e0[2], e0[3], pf[2]);
                    } else {
                        const float m1 = m[1] == NONE ? 0.f : m[1];
                        float sum1 = 0.f;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const bool dead = !inside && e1[x] == NONE;
                            const float e = exp2_fast(e1[x] - m1);
                            sum1 += e;
                            e1[x] = dead ? 0.f : e * frac;
                        }
                        l[1] = fmaf(sum1, unit[1], l[1]);
                        pf[1] = pack_half2(e1[0], e1[1]);
                        pf[3] = pack_half2(e1[2], e1[3]);
                    }
                    if (TWO) {
                        pl[0] = rest_half2(e0[0], e0[1], pf[0]);
                        pl[1] = rest_half2(e1[0], e1[1], pf[1]);
                        pl[2] = rest_half2(e0[2], e0[3], pf[2]);
                        pl[3] = rest_half2(e1[2], e1[3], pf[3]);
                    }
                }
                // ---- values: lane's tokens 2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4, columns D/8 g ..
                uint32_t vw[4][D / 32];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = warp * 16 + (x >> 1) * 8 + 2 * t4 + (x & 1);
                    if constexpr (D == 128) {
                        const uint4 u = *reinterpret_cast<const uint4*>(sm.v[stage] + row * D + (g ^ (row & 7)) * 16);
                        vw[x][0] = u.x, vw[x][1] = u.y, vw[x][2] = u.z, vw[x][3] = u.w;
                    } else {
                        const uint2 u = *reinterpret_cast<const uint2*>(
                            sm.v[stage] + row * D + ((g >> 1) ^ ((row >> 1) & 3)) * 16 + (g & 1) * 8);
                        vw[x][0] = u.x, vw[x][1] = u.y;
                    }
                }
#pragma unroll
                for (int x = 0; x < D / 32; ++x) {
                    const uint32_t l01 = __byte_perm(vw[0][x], vw[1][x], 0x5140), h01 = __byte_perm(vw[0][x], vw[1][x], 0x7362);
                    const uint32_t l23 = __byte_perm(vw[2][x], vw[3][x], 0x5140), h23 = __byte_perm(vw[2][x], vw[3][x], 0x7362);
                    const uint32_t b0[4] = {kv8_pair<0>(l01), kv8_pair<2>(l01), kv8_pair<0>(h01), kv8_pair<2>(h01)};
                    const uint32_t b1[4] = {kv8_pair<0>(l23), kv8_pair<2>(l23), kv8_pair<0>(h23), kv8_pair<2>(h23)};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        // (volatile, as the fence is: the values are used up before their stage goes)
                        mma_16816(acc[4 * x + y], pf, b0[y], b1[y], acc[4 * x + y]);
                        if (TWO) mma_16816(acc[4 * x + y], pl, b0[y], b1[y], acc[4 * x + y]);
                    }
                }
            }
            fence_proxy_async_shared();                      // the stage is refilled through the async proxy
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.empty[stage]);
            if (++stage == STAGES) stage = 0, phase ^= 1;
        }

        // ---- the four warps' sums, in the order of the warps; columns NT n + c, c < NT / 2, then the others
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
            l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
            l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
            if (t4 == 0) {
                sm.m[warp][g + 8 * half] = m[half];
                sm.l[warp][g + 8 * half] = l[half];
                sm.n[warp][g + 8 * half] = n[half];
            }
        }
        const bool whole = run == w.count;
        float* part = parts + ((size_t)cta * 2 + (ch == 0 ? 1 : 0)) * kv8_part_floats(RM, D);
        constexpr int HN = NT / 2, LD = D / 2 + 4;
#pragma unroll
        for (int cols = 0; cols < 2; ++cols) {
#pragma unroll
            for (int half = 0; half < HALVES; ++half)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int c = 0; c < HN; c += 4) {
                        float4 o;
                        float* po = reinterpret_cast<float*>(&o);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float* v = acc[cols * HN + c + y];
                            po[y] = SPLIT ? v[x] + v[2 + x] : v[2 * half + x];
                        }
                        *reinterpret_cast<float4*>(&sm.acc[warp][(g + 8 * half) * LD + (2 * t4 + x) * HN + c]) = o;
                    }
            if (cols == 0) {
                ok = !named_sync_or(!ok);
                if (!ok) break;
            } else {
                named_sync();
            }
            for (int i = tid; i < rows * (D / 8); i += WARPS * 32) {
                const int r = i / (D / 8), c = i % (D / 8) * 4, col = c / HN * NT + cols * HN + c % HN;
                float top = sm.m[0][r], top_n = sm.n[0][r];
#pragma unroll
                for (int k = 1; k < WARPS; ++k) top = fmaxf(top, sm.m[k][r]), top_n = fmaxf(top_n, sm.n[k][r]);
                float sum = 0.f;
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < WARPS; ++k) {
                    const float f = kv8_factor(sm.m[k][r], top);
                    sum = fmaf(sm.l[k][r], kv8_factor(sm.n[k][r], top_n), sum);
                    const float4 u = *reinterpret_cast<const float4*>(&sm.acc[k][r * LD + c]);
                    o.x = fmaf(u.x, f, o.x);
                    o.y = fmaf(u.y, f, o.y);
                    o.z = fmaf(u.z, f, o.z);
                    o.w = fmaf(u.w, f, o.w);
                }
                if (whole) {
                    int64_t at_lse;
                    T* dst = static_cast<T*>(a.out) + kv8_out_row(a, w.q.q0, head, tile * RM + r, &at_lse) + col;
                    const float inv = kv8_inverse(top, top_n, sum);
                    dst[0] = kv8_round<T>(o.x * inv);
                    dst[1] = kv8_round<T>(o.y * inv);
                    dst[2] = kv8_round<T>(o.z * inv);
                    dst[3] = kv8_round<T>(o.w * inv);
                    if (col == 0 && a.lse) a.lse[at_lse] = kv8_lse(top_n, sum);
                } else {
                    *reinterpret_cast<float4*>(part + 3 * RM + r * D + col) = o;
                    if (col == 0) part[r] = top, part[RM + r] = sum, part[2 * RM + r] = top_n;
                }
            }
            named_sync();
        }
        if (!ok) break;
        if (!whole && at == 0)
            // the rows' other pieces: as many CTAs as the rest of their chunks reaches into
            joint = Kv8Joint{w.s, head, tile, cut.of(w.pos + EXTRA + w.count - 1) - cta + 1};
        w.pos += take;
    }
    if (tid == 0) joints[cta] = ok ? joint : Kv8Joint{0, 0, 0, 0};
}

// Two CTAs a SM, and none that could never have a chunk.
int grid_of(const Kv8Attention& a) {
    const double most = (double)a.c.seqs * a.c.H * (((int64_t)a.c.width << a.c.logB) / CT + 1) * (((int64_t)a.c.T * a.G + 7) / 8);
    const int full = CTAS * kv8_sm_count();
    return most < full ? (int)most : full;
}

template <class T, int D, bool SPLIT>
cudaError_t run(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(kv8_stream_kernel<T, D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Shared<D>));
    if (e != cudaSuccess) return e;
    constexpr int RM = SPLIT ? 8 : 16;
    const int grid = grid_of(a);
    float* parts = static_cast<float*>(scratch);
    Kv8Joint* joints = reinterpret_cast<Kv8Joint*>(parts + (size_t)grid * 2 * kv8_part_floats(RM, D));
    g_launched.store(true, std::memory_order_release);
    e = launch_pdl(kv8_stream_kernel<T, D, SPLIT>, dim3(grid), dim3(THREADS), sizeof(Shared<D>), st, a, parts, joints);
    if (e != cudaSuccess) return e;
    // Few tiles of rows leave each of them many pieces: eight warps a row where there are at most a twelfth as many tiles
    // as CTAs (4 heads of 128, G = 8, bf16, us with eight and four: 1 sequence of 131072 tokens 38 and 41, 4 of 32768 16
    // and 18.5, 8 of 16384 21 and 20; 64 of up to 8192, 8 heads, 108 and 105).  What is counted is a bound, the
    // tokens of all sequences and a part-full tile of each: one decoded token a sequence with G >= RM counts twice.
    const int64_t tiles = (int64_t)a.c.H * ((int64_t)a.c.T * a.G / RM + a.c.seqs);
    const Kv8Joint* j = joints;
    const float* p = parts;
    if (tiles <= grid / 12)
        return launch_pdl(kv8_join_kernel<T, D, RM, 8>, dim3(grid, RM), dim3(KV8_JOIN_WARPS * 32), 0, st, a, p, j);
    return launch_pdl(kv8_join_kernel<T, D, RM, 4>, dim3(grid, RM / 2), dim3(KV8_JOIN_WARPS * 32), 0, st, a, p, j);
}

template <class T, bool SPLIT>
cudaError_t run_d(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    return a.c.D == 64 ? run<T, 64, SPLIT>(a, scratch, st) : run<T, 128, SPLIT>(a, scratch, st);
}

}  // namespace

size_t kv8_stream_scratch(const Kv8Attention& a) {
    return (size_t)grid_of(a) * (2 * kv8_part_floats(16, a.c.D) * sizeof(float) + sizeof(Kv8Joint));
}

cudaError_t launch_kv8_stream(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    if (a.dtype == TQ2_F32) return run_d<float, true>(a, scratch, st);
    if (a.dtype == TQ2_F16) return a.narrow ? run_d<__half, true>(a, scratch, st) : run_d<__half, false>(a, scratch, st);
    return run_d<__nv_bfloat16, false>(a, scratch, st);
}

unsigned int read_clear_dev_error_kv8_stream(cudaStream_t st) { return read_clear_record(st); }

}  // namespace tq2
