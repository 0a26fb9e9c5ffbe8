// kv8_umma.cu -- attention of many rows over the 8-bit cache on tcgen05: prompts,
// chunks of prompts, an encoder's states.
//
// Mathematics: as the streaming path (kv8_stream.cu), with the whole weight
// 2^(w_t - m), w_t = (scale log2(e) ks) (q . c) + log2 vs, in f16, and
// l = sum 2^(w_t - m) 2^x / vs, x the exponent of the first vs (blocks of zeros: vs 2^(x - 40) in both).  ks and vs are constant over 16 columns, so per score that is
// half a packed multiply-add, one exponential and half a packed sum.  Where a vs is too far from 2^x for
// that, a piece's weights have a sum (and exponentials) of their own from there on.
//
// A CTA takes 256 rows (f32: 128), a row being a query token and one of the heads
// that share a head of the cache, over tiles of 128 tokens.  Warps: one brings packed
// tiles by TMA, four decode them (code - 128, exact in f16) into the swizzled layout of the MMAs'
// operands, one issues S = Q K^T (both from shared memory) and O += P V (P from tensor
// memory, over S's columns), a group of four for every 128 rows does the softmax, a
// thread a row, while the MMAs work for the other group, and one walks the list of what is to be
// done.  f32 queries are two f16 parts, f32 and f16 results' weights too (twice the MMAs of that
// product: with one part, a weight's rounding is as large as an f16 result's own).  All tiles of
// all rows are cut over the CTAs by what they cost; what a cut divides is joined afterwards.
//
// The MMAs are issued in the order Q K^T, P V, Q K^T .. of a group, and execute in that order: P V
// reads P before the next scores take its place, and scores that are there mean that the
// last P V is done, so the group may rescale O.
//
// Bound: 8192 causal tokens, 8 heads of 128, G = 4, bf16: 533 us, 1.03 PFLOP/s (53 % of the measured
// peak; tensor pipe 46 %, issue slots 52 %; f16, with two parts of each weight, 672, f32, with two of queries too and half
// the rows a CTA, 1326).  A tile of 128 x 256 takes 4100 cycles, its MMAs 2048.  A group's
// scores, softmax and values follow one another (2 x 512 cycles of MMAs, 600 until their completion is seen,
// 1700 of softmax beside the other group's and the decoders), and the operands' reads, the decoders' and the copies
// want shared memory for 2500 of the 4100.  Sums of their own, where scales are 2^40 apart, take twice the time (1110).
// What the instruction cache does not hold costs time in every role, so code that runs once a tile is kept in short loops,
// and what runs once a piece is read from one list.  (The code of sums of their own, which such calls never run, costs 2 %;
// a reference of its own for every row's sum cost 5 to 9.)
#include <cfloat>
#include <type_traits>

#include "kv8_join.cuh"
#include "q4.cuh"

namespace tq2 {
namespace {

constexpr int KT = 128;         // tokens of a tile
constexpr int THREADS = 512;
constexpr int DECODERS = 4;     // warps
constexpr int BUFS = 4;         // decoded tiles: keys and values in turn
constexpr int CONS = 4;         // tiles whose scales are at hand
// The cut counts a tile of rows as its tiles of tokens and so many more, which is about what queries, masked tiles and
// the result cost.  A cut through those is one at their start.
constexpr int EXTRA = 4;
constexpr int LEAST = EXTRA + 1;                             // units of a CTA: no two cuts through the same EXTRA
constexpr float HEAD = 6.f, RAISE = 14.f;                    // as kv8_stream.cu
constexpr float TINY = 0x1p-103f;
constexpr uint32_t S_COL = 0, O_COL = 256;                  // columns of tensor memory: scores, sums

template <class T, int D>
struct Form {
    static constexpr bool SPLIT = sizeof(T) == 4;
    static constexpr bool TWO = !std::is_same<T, __nv_bfloat16>::value;   // parts of a weight
    static constexpr int NQ = SPLIT ? 1 : 2;                 // groups of 128 rows
    static constexpr int ROWS = NQ * 128;
    static constexpr int RAW = D == 128 ? 2 : 6;             // packed tiles
    static constexpr int SLAB = KT * 128;                    // 128 rows of 64 f16
    static constexpr int TILE = SLAB * (D / 64);             // 128 rows of D f16
};

// Tiles of one tile of rows in a row: what a CTA's roles work on between two results.  (One warp walks the list and says
// what is next, so that the others hold no more than this.)
struct Piece {
    int s, head, tile, rows;    // rows: of the sequence's head
    int q0, n, len, first;      // first tile of 128 tokens
    int run, whole, part;       // tiles; whether they are all of the rows'; else the part that takes the sums
    int pad;
};
constexpr int PIECES = 4;

template <class T, int D>
struct __align__(1024) Shared {
    uint8_t q[2][Form<T, D>::TILE];                          // by group (f32: by part)
    uint8_t kv[BUFS][Form<T, D>::TILE];
    uint8_t raw[Form<T, D>::RAW][KT * D];
    float4 cons[CONS][KT / 16];                              // ks, log2 vs, 2^x / vs; w: values count (NaN: are no numbers)
    int near[CONS];                                          // 4 x, and 0: all vs of the piece so far are near it, 1: now not, 2: no more
    float2 scales[CONS][8];                                  // of keys and values, by piece; -1: nothing there
    uint64_t raw_full[Form<T, D>::RAW], raw_empty[Form<T, D>::RAW];
    uint64_t kv_full[BUFS], kv_empty[BUFS], cons_full[CONS];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2], idle;
    Piece pieces[PIECES];                                    // run 0: no more
    uint64_t piece_full[PIECES], piece_empty[PIECES];
    long long sums[THREADS / 32];
    uint32_t tmem;
    int seq, head, tile, at;
    volatile int abort;
};

// Rows of one head of a sequence in tiles of ROWS, and the KV tiles each of them goes over.
struct Seq {
    Kv8Seq q;
    int rows, tiles;
};
template <int ROWS>
__device__ __forceinline__ Seq seq_of(const Kv8Attention& a, int s) {
    Seq r;
    r.q = kv8_seq(a.c, s);
    r.rows = r.q.n * a.G;
    r.tiles = r.rows <= a.few ? 0 : (r.rows + ROWS - 1) / ROWS;
    return r;
}
// First tile of 128 tokens that some row of a tile sees, and the number of them (at least one).
template <int ROWS>
__device__ __forceinline__ int2 span_of(const Kv8Attention& a, const Seq& s, int tile) {
    const int r0 = tile * ROWS, r1 = min(r0 + ROWS, s.rows) - 1, p = s.q.len - s.q.n;
    const int hi = a.causal ? min(s.q.len, p + r1 / a.G + 1) : s.q.len;
    const int lo = a.window ? max(p + r0 / a.G - a.window + 1, 0) : 0;
    const int first = lo / KT;
    return make_int2(first, max((hi + KT - 1) / KT - first, 1));
}

// Units of one head of a lane's own sequence s (0 where there is none).
template <int ROWS>
__device__ __forceinline__ long long lane_units(const Kv8Attention& a, int s, int end, Seq& q, int lane) {
    long long u = 0;
    q.tiles = 0;
    if (s < end) q = seq_of<ROWS>(a, s);
    const bool many = q.tiles > 4;
    if (!many)
#pragma unroll 1
        for (int t = 0; t < q.tiles; ++t) u += span_of<ROWS>(a, q, t).y + EXTRA;
#pragma unroll 1
    for (uint32_t rest = __ballot_sync(0xffffffffu, many); rest; rest &= rest - 1) {
        const int owner = __ffs(rest) - 1;
        const Seq o = seq_of<ROWS>(a, __shfl_sync(0xffffffffu, s, owner));
        long long sum = 0;
#pragma unroll 1
        for (int t = lane; t < o.tiles; t += 32) sum += span_of<ROWS>(a, o, t).y + EXTRA;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == owner) u = sum;
    }
    return u;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += u;
    }
    return v;
}

using F2 = unsigned long long;  // two f32
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 f2_parts(F2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max16(const uint32_t* v) {
    auto f = [&](int i) { return __uint_as_float(v[i]); };
    const float a = max3(f(0), f(1), f(2)), b = max3(f(3), f(4), f(5)), c = max3(f(6), f(7), f(8));
    const float d = max3(f(9), f(10), f(11)), e = max3(f(12), f(13), f(14));
    return max3(max3(a, b, c), max3(d, e, f(15)), kv8_none());
}

// Scores are read from tensor memory twice (64 columns take 50 cycles) rather than held: the loops stay short, which
// the instruction caches of warps in four different roles ask for.

// The largest exponent of a row's 128 weights, all of them seen.
__device__ __forceinline__ float tile_top(uint32_t s_addr, const float4* cons, float qa) {
    float t = kv8_none();
#pragma unroll 1
    for (int c = 0; c < KT; c += 64) {
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(s_addr + c, v[0]);
        tmem_ld_32x32b_x32(s_addr + c + 32, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const float4 k = cons[c / 16 + h];
            t = fmaxf(t, fmaf(max16(&v[h >> 1][16 * (h & 1)]), k.x * qa, k.y));
        }
    }
    return t;
}

// The sum of a row's weights, with a reference n of their own.  The scores are as they came (raw), or the weights' exponents
// with -Inf in columns that the row does not see.
__device__ __forceinline__ void tile_sum(uint32_t s_addr, const float4* cons, float qa, bool raw, float& l, float& n) {
    float top = kv8_none();
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {                   // their largest, then their sum
        const float ref = n == kv8_none() ? 0.f : n;
#pragma unroll 1
        for (int c = 0; c < KT; c += 16) {
            const float4 k = cons[c / 16];
            if (k.y == kv8_none()) continue;
            uint32_t v[16];
            tmem_ld_32x32b_x16(s_addr + c, v);
            tmem_wait_ld();
            const float ks = raw ? k.x * qa : 1.f, off = raw ? 0.f : -k.y;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const float z = fmaf(__uint_as_float(v[e]), ks, off);
                if (pass) l += exp2_fast(z - ref);
                else top = fmaxf(top, z);
            }
        }
        if (!pass && top > n + RAISE) {
            l *= exp2_fast(n - (top - HEAD));
            n = top - HEAD;
        }
        __syncwarp();
    }
}

// NaN in place of the weights' exponents of seen tokens whose values are no numbers (raw: of all of them).
__device__ __forceinline__ void tile_poison(uint32_t s_addr, const float4* cons, bool raw) {
#pragma unroll 1
    for (int c = 0; c < KT; c += 16) {
        if (!isnan(cons[c / 16].w)) continue;
        uint32_t v[16];
        tmem_ld_32x32b_x16(s_addr + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (raw || __uint_as_float(v[e]) != kv8_none()) v[e] = 0x7fffffffu;
        tmem_st_32x32b_x16(s_addr + c, v);
    }
    tmem_wait_st();
}

// Weights of 2 N tokens relative to a reference: f16 pairs (and what those leave), added to sum.
template <bool TWO, int N>
__device__ __forceinline__ F2 weights_of(const uint32_t* v, F2 ks, F2 off, uint32_t* ph, uint32_t* pl) {
    F2 sum = f2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const float2 x = f2_parts(f2_fma(f2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])), ks, off));
        const float e0 = exp2_fast(x.x), e1 = exp2_fast(x.y);
        sum = f2_add(sum, f2(e0, e1));
        ph[e] = pack_half2(e0, e1);
        if (TWO) pl[e] = rest_half2(e0, e1, ph[e]);
    }
    return sum;
}

// The row's weights relative to ref, in place of its scores: 32 tokens' are 16 columns (and 16 of second
// parts).  Returns l with their sum.
template <bool TWO>
__device__ __forceinline__ float tile_weights(uint32_t s_addr, const float4* cons, float qa, float ref, float l) {
#pragma unroll 1
    for (int c = 0; c < KT; c += 64) {
        uint32_t v[2][32];
        tmem_ld_32x32b_x32(s_addr + c, v[0]);
        tmem_ld_32x32b_x32(s_addr + c + 32, v[1]);
        tmem_wait_ld();
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            uint32_t ph[16], pl[16];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 k = cons[c / 16 + 2 * g + h];
                const float ks = k.x * qa, off = k.y - ref;
                const float2 both = f2_parts(weights_of<TWO, 8>(&v[g][16 * h], f2(ks, ks), f2(off, off), ph + 8 * h, pl + 8 * h));
                l = fmaf(both.x + both.y, k.z, l);
            }
            tmem_st_32x32b_x16(s_addr + c + 32 * g, ph);
            if (TWO) tmem_st_32x32b_x16(s_addr + c + 32 * g + 16, pl);
        }
    }
    return l;
}

// Both for tiles of which the row sees columns lo .. hi-1 alone.  (Scores become exponents in their place first.)
__device__ __forceinline__ float tile_top_some(uint32_t s_addr, const float4* cons, float qa, int lo, int hi) {
    float t = kv8_none();
    lo = max(lo, 0);
#pragma unroll 1
    for (int c = 0; c < KT; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(s_addr + c, v);
        tmem_wait_ld();
        const uint32_t from = lo - c, count = max(hi - lo, 0);       // column e is seen: e - from < count
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4 k = cons[c / 16 + h];
            const float ks = k.x * qa;
#pragma unroll
            for (int e = 16 * h; e < 16 * h + 16; ++e)
                v[e] = __float_as_uint(e - from < count ? fmaf(__uint_as_float(v[e]), ks, k.y) : kv8_none());
            t = fmaxf(t, max16(v + 16 * h));
        }
        tmem_st_32x32b_x32(s_addr + c, v);
    }
    tmem_wait_st();
    return t;
}
template <bool TWO>
__device__ __forceinline__ float tile_weights_some(uint32_t s_addr, const float4* cons, float ref, float l) {
#pragma unroll 1
    for (int c = 0; c < KT; c += 32) {
        uint32_t v[32], ph[16], pl[16];
        tmem_ld_32x32b_x32(s_addr + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 both = f2_parts(weights_of<TWO, 8>(v + 16 * h, f2(1.f, 1.f), f2(-ref, -ref), ph + 8 * h, pl + 8 * h));
            l = fmaf(both.x + both.y, cons[c / 16 + h].z, l);
        }
        tmem_st_32x32b_x16(s_addr + c, ph);
        if (TWO) tmem_st_32x32b_x16(s_addr + c + 16, pl);
    }
    return l;
}

// A warp's 32 rows of queries, scaled by a power of two to 2^14 .. 2^15, in the layout of an MMA operand (the scores of
// the rows before are there, so nobody reads those any more).  Returns the power of the lane's row.  Raw pieces
// of 8 elements are copied to where their f16 values (f32: first and second parts) go, and converted in place.
// A row that has a NaN or Inf becomes zeros, and its power NO_NUMBERS: it is NaN at the end if it saw a token.
constexpr int NO_NUMBERS = 1 << 20;
template <class T, int D>
__device__ __forceinline__ int load_queries(const Kv8Attention& a, Shared<T, D>& sm, const Piece& w, int qi,
                                            int warp, int lane) {
    using F = Form<T, D>;
    constexpr int LPR = D / 8, RPP = 32 / LPR;               // lanes a row, rows a pass
    const int el = lane % LPR * 8, r0 = w.tile * F::ROWS + qi * 128 + warp * 32;
    const int i0 = warp * 32 + lane / LPR;                   // of the group
    uint8_t* const to0 = sm.q[F::SPLIT ? 0 : qi] + (el / 64) * F::SLAB;
    auto place = [&](int i) { return to0 + i * 128 + (el % 64 / 8 ^ (i & 7)) * 16; };
    const T* const q = static_cast<const T*>(a.q) + (int64_t)w.q0 * a.qt + (int64_t)w.head * a.G * a.qh + el;
    auto row_of = [&](int pass) {                            // (rows that are none: the last one, cleared below)
        const int r = min(r0 + lane / LPR + pass * RPP, w.rows - 1), token = r / a.G;
        return q + token * a.qt + (r - token * a.G) * a.qh;
    };
    if (a.qvec) {
#pragma unroll 4
        for (int pass = 0; pass < LPR; ++pass) {
            const T* p = row_of(pass);
            uint8_t* to = place(i0 + pass * RPP);
            cp_async16(to, p);
            if (F::SPLIT) cp_async16(to + F::TILE, p + 4);
        }
    } else {
#pragma unroll 1
        for (int pass = 0; pass < LPR; ++pass) {
            const T* p = row_of(pass);
            uint8_t* to = place(i0 + pass * RPP);
#pragma unroll 1
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<T*>(to + (F::SPLIT ? k / 4 * F::TILE + k % 4 * 4 : k * 2)) = p[k];
        }
    }
    cp_async_wait_all();
    int power = 0;
    constexpr int DEEP = 4;                                  // passes side by side
#pragma unroll 1
    for (int p0 = 0; p0 < LPR; p0 += DEEP) {
        uint4 raw[DEEP][F::SPLIT ? 2 : 1];
        uint32_t most[DEEP];
        int e[DEEP];
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            uint8_t* to = place(i0 + (p0 + d) * RPP);
            const bool live = r0 + lane / LPR + (p0 + d) * RPP < w.rows;
            raw[d][0] = live ? *reinterpret_cast<const uint4*>(to) : make_uint4(0, 0, 0, 0);
            if constexpr (F::SPLIT) raw[d][1] = live ? *reinterpret_cast<const uint4*>(to + F::TILE) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const T* u = reinterpret_cast<const T*>(raw[d]);
            most[d] = 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) most[d] = max(most[d], __float_as_uint(kv8_wide(u[k])) & 0x7fffffffu);
        }
#pragma unroll
        for (int k = 1; k < LPR; k <<= 1)
#pragma unroll
            for (int d = 0; d < DEEP; ++d) most[d] = max(most[d], __shfl_xor_sync(0xffffffffu, most[d], k));
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            e[d] = most[d] < 0x7f800000u ? kv8_power(__uint_as_float(most[d])) : NO_NUMBERS;
            const int of = __shfl_sync(0xffffffffu, e[d], (lane - (p0 + d) * RPP) * LPR & 31);
            if (lane / RPP == p0 + d) power = of;
        }
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            const T* u = reinterpret_cast<const T*>(raw[d]);
            const bool numbers = e[d] != NO_NUMBERS;
            const float up = copysignf(__uint_as_float((uint32_t)(e[d] + 127) << 23), a.scale);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float x0 = numbers ? kv8_wide(u[2 * k]) * up : 0.f, x1 = numbers ? kv8_wide(u[2 * k + 1]) * up : 0.f;
                hi[k] = pack_half2(x0, x1);
                if (F::SPLIT) lo[k] = rest_half2(x0, x1, hi[k]);
            }
            uint8_t* to = place(i0 + (p0 + d) * RPP);
            *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            if constexpr (F::SPLIT) *reinterpret_cast<uint4*>(to + F::TILE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_full[qi]);
    return power;
}

// A row of O times inv to its place in global memory.
template <class T, int D>
__device__ __forceinline__ void store_row(uint32_t o_addr, bool live, float inv, T* out) {
    if (__any_sync(0xffffffffu, reinterpret_cast<uintptr_t>(out) & 15)) {
#pragma unroll 1
        for (int c = 0; c < D; c += 2) {
            uint32_t v[2];
            tmem_ld_32x32b_x2(o_addr + c, v);
            tmem_wait_ld();
            if (live) out[c] = kv8_round<T>(__uint_as_float(v[0]) * inv), out[c + 1] = kv8_round<T>(__uint_as_float(v[1]) * inv);
        }
        return;
    }
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        uint32_t v[16];
        float y[16];
        tmem_ld_32x32b_x16(o_addr + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(v[e]) * inv;
        if (live) kv8_store16(out + c, true, y);
    }
}

// The MMAs of one group: scores S = Q K^T, and values O (+)= P V.
template <class F, int D>
__device__ __forceinline__ void issue_scores(uint32_t s, uint64_t q, uint64_t k) {
    constexpr uint32_t idesc = idesc_f16_f32(128, KT);
#pragma unroll
    for (int part = 0; part < (F::SPLIT ? 2 : 1); ++part)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = ((i >> 2) * F::SLAB + (i & 3) * 32) >> 4;
            umma_f16_ss(s, q + (part * F::TILE >> 4) + off, k + off, idesc, part || i);
        }
}
template <class F, int D>
__device__ __forceinline__ void issue_values(uint32_t o, uint32_t p, uint64_t v, uint32_t add) {
    constexpr uint32_t idesc = idesc_f16_f32_bmn(128, D);
#pragma unroll
    for (int i = 0; i < KT / 16; ++i)
#pragma unroll
        for (int part = 0; part < (F::TWO ? 2 : 1); ++part)
            umma_f16_ts(o, p + 32 * (i >> 1) + 16 * part + 8 * (i & 1), v + (i * 2048 >> 4), idesc, i || part ? 1u : add);
}

template <class T, int D>
__global__ void __launch_bounds__(THREADS, 1)
kv8_umma_kernel(const __grid_constant__ Kv8Attention a, float* parts, Kv8Joint* joints) {
    using F = Form<T, D>;
    constexpr int ROWS = F::ROWS;
    extern __shared__ __align__(1024) uint8_t raw_shared[];
    Shared<T, D>& sm = *reinterpret_cast<Shared<T, D>*>(raw_shared);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < F::RAW; ++i) {
            mbar_init(&sm.raw_full[i], 33);
            mbar_init(&sm.raw_empty[i], DECODERS);
        }
        for (int i = 0; i < BUFS; ++i) {
            mbar_init(&sm.kv_full[i], DECODERS);
            mbar_init(&sm.kv_empty[i], 1);
        }
        for (int i = 0; i < CONS; ++i) mbar_init(&sm.cons_full[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 4);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 4);
            mbar_init(&sm.o_full[i], 1);
        }
        for (int i = 0; i < PIECES; ++i) {
            mbar_init(&sm.piece_full[i], 1);
            mbar_init(&sm.piece_empty[i], 2 + DECODERS + 4 * F::NQ);
        }
        mbar_init(&sm.idle, 1);
        sm.abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&a.map);
    }
    pdl_launch_dependents();
    pdl_wait();

    // the whole list's length (a head's times H), and where this CTA's share begins
    const int S = a.c.seqs, per = (S + THREADS / 32 - 1) / (THREADS / 32);
    const int slice_end = min((warp + 1) * per, S);
    long long mine = 0;
    Seq q;
#pragma unroll 1
    for (int s = warp * per; s < slice_end; s += 32) mine += lane_units<ROWS>(a, s + lane, slice_end, q, lane);
#pragma unroll
    for (int d = 16; d; d >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, d);
    mine *= a.c.H;
    if (lane == 0) sm.sums[warp] = mine;
    __syncthreads();
    long long total = 0, before = 0;
    for (int i = 0; i < THREADS / 32; ++i) {
        if (i < warp) before += sm.sums[i];
        total += sm.sums[i];
    }
    const Kv8Cut cut(total, gridDim.x, LEAST);
    const int cta = blockIdx.x;
    if (cta >= cut.ctas) {
        if (tid == 0) joints[cta].pieces = 0;
        return;
    }
    const long long begin = cut.begin(cta);
    if (before <= begin && begin < before + mine) {
#pragma unroll 1
        for (int s = warp * per; s < slice_end; s += 32) {
            const long long u = lane_units<ROWS>(a, s + lane, slice_end, q, lane);
            const long long incl = warp_scan(u * a.c.H, lane);
            const uint32_t past = __ballot_sync(0xffffffffu, before + incl > begin);
            if (!past) {
                before += __shfl_sync(0xffffffffu, incl, 31);
                continue;
            }
            const int owner = __ffs(past) - 1;
            const long long in = begin - before - __shfl_sync(0xffffffffu, incl - u * a.c.H, owner);
            const long long uh = __shfl_sync(0xffffffffu, u, owner);
            q = seq_of<ROWS>(a, s + owner);
            long long left = in % uh;
#pragma unroll 1
            for (int t = 0;; t += 32) {
                const long long c = t + lane < q.tiles ? span_of<ROWS>(a, q, t + lane).y + EXTRA : 0;
                const long long sum = warp_scan(c, lane);
                const uint32_t there = __ballot_sync(0xffffffffu, sum > left);
                if (!there) {
                    left -= __shfl_sync(0xffffffffu, sum, 31);
                    continue;
                }
                const int o = __ffs(there) - 1;
                left -= __shfl_sync(0xffffffffu, sum - c, o);
                if (lane == 0) {
                    sm.seq = s + owner;
                    sm.head = (int)(in / uh);
                    sm.tile = t + o;
                    sm.at = (int)left;
                }
                break;
            }
            break;
        }
    }
    if (warp == 2) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = 0;
    volatile int* abort_flag = &sm.abort;
    const int logB = a.c.logB, rows_piece = min(1 << logB, KT / 2), pieces = KT / rows_piece;

    // a role's next piece, and its leave of it
    uint32_t pieces_seen = 0;
    auto next_piece = [&](Piece& w) {
        const int slot = pieces_seen & (PIECES - 1);
        if (!kv8_wait(&sm.piece_full[slot], pieces_seen / PIECES & 1, abort_flag, true)) return false;
        w = sm.pieces[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.piece_empty[slot]);
        ++pieces_seen;
        return w.run > 0;
    };

    if (warp == 3) {                                         // ---- the list
        int s = sm.seq, head = sm.head, tile = sm.tile, at = sm.at;      // at: units of the rows that are behind
        long long pos = begin;
        const long long end = cut.begin(cta + 1);
        if (at <= EXTRA) pos -= at, at = 0;
        Seq q = seq_of<ROWS>(a, s);
        Kv8Joint joint{0, 0, 0, 0};
        for (uint32_t i = 0;; ++i) {
            const int slot = i & (PIECES - 1);
            if (!kv8_wait(&sm.piece_empty[slot], (i / PIECES & 1) ^ 1, abort_flag, true)) {
                joint.pieces = 0;
                break;
            }
            const int2 span = span_of<ROWS>(a, q, tile);
            const int take = (int)min((long long)(span.y + EXTRA - at), end - pos);
            const int behind = max(at - EXTRA, 0), run = max(take - (at ? 0 : EXTRA), 0);
            if (lane == 0) {
                sm.pieces[slot] = Piece{s, head, tile, q.rows, q.q.q0, q.q.n, q.q.len, span.x + behind, run, run == span.y,
                                        at == 0 ? 1 : 0, 0};
                mbar_arrive(&sm.piece_full[slot]);
            }
            if (run == 0) break;
            if (run < span.y && at == 0)
                // the rows' other pieces: as many CTAs as the rest of their tiles reaches into
                joint = Kv8Joint{s, head, tile, cut.of(pos + EXTRA + span.y - 1) - cta + 1};
            pos += take;
            at = 0;                                          // (unless nothing is left, the piece ended its rows)
            if (pos < end && ++tile == q.tiles) {
                tile = 0;
                if (++head == a.c.H) {
                    head = 0;
                    do q = seq_of<ROWS>(a, ++s);
                    while (q.tiles == 0);
                }
            }
        }
        if (lane == 0) joints[cta] = joint;
    } else if (warp == 0) {                                  // ---- packed tiles
        Piece w;
        int st = 0;
        uint32_t ph = 0;
        uint32_t g = 0;
        bool wrapped = false, ok = true;
        fence_proxy_async_shared();
        asm volatile("fence.proxy.async.global;" ::: "memory");
        while (ok && next_piece(w)) {
            const int from = a.window ? max(w.len - w.n - a.window + 1, 0) : 0;
            for (int i = 0; ok && i < w.run; ++i, ++g) {
                const int token = (w.first + i) * KT + lane * rows_piece;
                int block = -1;
                if (lane < pieces && token < w.len && token + rows_piece > from) block = kv8_block(a.c, w.s, token);
                const uint32_t here = __ballot_sync(0xffffffffu, block >= 0);
                const int inside = token & ((1 << logB) - 1);
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    if (!kv8_wait(&sm.raw_empty[st], ph ^ 1, abort_flag, true)) {
                        ok = false;
                        break;
                    }
                    if (kv == 0) {
                        float2* sc = &sm.scales[g & (CONS - 1)][lane & 7];
                        if (block >= 0) {
                            const float* src = a.c.scales + (int64_t)block * 2 * a.c.H + w.head;
                            cp_async4(&sc->x, src);
                            cp_async4(&sc->y, src + a.c.H);
                        } else if (lane < pieces) {
                            *sc = make_float2(0.f, -1.f);
                        }
                    }
                    __syncwarp();                            // the ordinary stores are lane 0's to release
                    if (lane == 0) mbar_arrive_expect_tx(&sm.raw_full[st], __popc(here) * (uint32_t)(rows_piece * D));
                    if (block >= 0)
                        tma_load_2d(sm.raw[st] + lane * rows_piece * D, &a.map, &sm.raw_full[st], 0,
                                    (int)(kv8_row(a.c, block, kv, w.head) + inside));
                    cp_async_arrive(&sm.raw_full[st]);
                    if (++st == F::RAW) st = 0, ph ^= 1, wrapped = true;
                }
            }
        }
        if (!ok)                                             // copies in flight end before the shared memory goes
            for (int u = 0; u < F::RAW; ++u)
                if (u < st || wrapped) mbar_wait(&sm.raw_full[u], u < st ? ph : ph ^ 1);
    } else if (warp == 1) {                                  // ---- MMA issuer
        const uint64_t q0_desc = sdesc_kmajor_sw128(smem_u32(sm.q[0])), k0_desc = sdesc_kmajor_sw128(smem_u32(sm.kv[0]));
        const uint64_t v0_desc = sdesc_mnmajor_sw128(smem_u32(sm.kv[0]), F::SLAB, 1024);
        uint32_t q_ph = 0, p_ph = 0;                         // a bit a group
        uint32_t g = 0;                                      // tiles
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && kv8_wait(bar, parity, abort_flag, true); };
        Piece w;
        while (ok && __any_sync(0xffffffffu, next_piece(w))) {
            const int nq = __shfl_sync(0xffffffffu, w.rows - w.tile * ROWS > 128 ? F::NQ : 1, 0);
            const int run = __shfl_sync(0xffffffffu, w.run, 0);
            // step i: the values of tile i, and of each group right behind them the scores of tile i + 1
#pragma unroll 1
            for (int i = -1; ok && i < run; ++i) {
                const bool more = i + 1 < run;
                const int vb = (2 * g - 1) & 3, kb = 2 * g & 3;              // (g: tile i + 1 of all)
                const uint32_t v_ph = (g - 1) >> 1 & 1, k_ph = g >> 1 & 1;
#pragma unroll 1
                for (int qi = 0; qi < nq; ++qi) {
                    if (i >= 0) {
                        if (!wait(&sm.p_full[qi], p_ph >> qi & 1)) break;
                        p_ph ^= 1 << qi;
                        if (qi == 0 && !wait(&sm.kv_full[vb], v_ph)) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_values<F, D>(O_COL + D * qi, S_COL + 128 * qi, v0_desc + (uint32_t)vb * (F::TILE >> 4), i > 0);
                            if (qi == nq - 1) umma_commit(&sm.kv_empty[vb]);
                            if (!more) umma_commit(&sm.o_full[qi]);
                        }
                        __syncwarp();
                    } else {
                        if (!wait(&sm.q_full[qi], q_ph >> qi & 1)) break;
                        q_ph ^= 1 << qi;
                    }
                    if (more) {
                        if (qi == 0 && !wait(&sm.kv_full[kb], k_ph)) break;
                        tc_fence_after();
                        if (elect_one()) {
                            issue_scores<F, D>(S_COL + 128 * qi, q0_desc + (uint32_t)qi * (F::TILE >> 4),
                                               k0_desc + (uint32_t)kb * (F::TILE >> 4));
                            umma_commit(&sm.s_full[qi]);
                            if (qi == nq - 1) umma_commit(&sm.kv_empty[kb]);
                        }
                        __syncwarp();
                    }
                }
                if (more) ++g;
            }
        }
        if (!ok) {                                           // MMAs in flight end before their operands go
            if (elect_one()) umma_commit(&sm.idle);
            __syncwarp();
            mbar_wait(&sm.idle, 0);
        }
    } else if (warp >= 12) {                                 // ---- decoders: 32 tokens of a tile each
        const int dw = warp - 12;
        int st = 0;
        uint32_t ph = 0;
        bool ok = true;
        uint32_t g = 0;
        int x = 0, far = 0;
        Piece w;
        while (ok && next_piece(w))
        for (int i = 0; ok && i < w.run; ++i, ++g) {
            const int slot = g & (CONS - 1);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
                const int buf = (2 * g & 3) + kv;
                if (!kv8_wait(&sm.raw_full[st], ph, abort_flag, true) ||
                    !kv8_wait(&sm.kv_empty[buf], (g >> 1 & 1) ^ 1, abort_flag, true)) {
                    ok = false;
                    break;
                }
                if (kv == 0 && dw == 0) {
                    const int group = lane & (KT / 16 - 1);
                    float2 sc = sm.scales[slot][group * 16 / rows_piece];
                    if (!(sc.x <= FLT_MAX)) sc.x = __int_as_float(0x7fffffff);
                    const bool number = sc.y <= FLT_MAX, some = number && sc.y >= TINY;      // (values that are not all zeros)
                    const float y = some ? log2f(sc.y) : kv8_none();
                    if (i == 0) {
                        float most = y;
#pragma unroll
                        for (int d = 1; d < KT / 16; d <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
                        x = most == kv8_none() ? 0 : (int)fminf(floorf(most), 127.f);
                        far = 0;
                    }
                    far = far ? 2 : __any_sync(0xffffffffu, !number || (some && fabsf(y - x) > KV8_NEAR));
                    float4 c = make_float4(sc.x, y, exp2_fast((float)x) / sc.y, 1.f);
                    if (!some) c = make_float4(sc.x, x - KV8_NEAR, KV8_FAR, 0.f);        // zeros weigh, as little as counts
                    if (!number) c = make_float4(sc.x, (float)x, 1.f, __int_as_float(0x7fffffff));
                    if (sc.y < 0.f) c = make_float4(0.f, kv8_none(), 1.f, 0.f);          // no block: nobody sees it
                    if (lane < KT / 16) sm.cons[slot][lane] = c;
                    if (lane == 0) sm.near[slot] = 4 * x + far;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sm.cons_full[slot]);
                } else if (kv && !kv8_wait(&sm.cons_full[slot], g / CONS & 1, abort_flag, true)) {
                    ok = false;
                    break;
                }
                const uint8_t* src = sm.raw[st];
                uint8_t* dst = sm.kv[buf];
                // Eight rows of 64 packed bytes a step.  Lanes 0..3 and 4..7 of a phase take rows r and r ^ 5: their swizzled
                // 16-byte pieces lie in different halves of a line, and those of f16 in its even and odd pieces.
                constexpr int DEEP = 2;                      // steps whose loads are in flight
                const int in8 = (lane >> 3) ^ ((lane >> 2 & 1) * 5), c = lane & 3;
                const int row0 = dw * 32 + in8;
                const int from = row0 * D + (D == 128 ? c ^ in8 : c ^ (in8 >> 1 & 3)) * 16;
                const int to = row0 * 128 + (2 * c ^ in8) * 16;
                const bool any_zero = kv && __any_sync(0xffffffffu, lane < 2 && sm.cons[slot][dw * 2 + (lane & 1)].w == 0.f);
#pragma unroll 1
                for (int x0 = 0; x0 < D / 16; x0 += DEEP) {
                    uint4 u[DEEP];
#pragma unroll
                    for (int x = 0; x < DEEP; ++x) {
                        const int block = (x0 + x) & 3, slab = (x0 + x) >> 2;      // of 8 rows, of 64 columns
                        u[x] = *reinterpret_cast<const uint4*>(src + (from ^ (slab * 64)) + block * 8 * D);
                        if (any_zero && sm.cons[slot][dw * 2 + (block >> 1)].w == 0.f)
                            u[x] = make_uint4(0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u);
                    }
#pragma unroll
                    for (int x = 0; x < DEEP; ++x) {
                        const int block = (x0 + x) & 3, slab = (x0 + x) >> 2;
                        uint8_t* p = dst + slab * F::SLAB + block * 1024;
                        *reinterpret_cast<uint4*>(p + to) =
                            make_uint4(kv8_pair<0>(u[x].x), kv8_pair<2>(u[x].x), kv8_pair<0>(u[x].y), kv8_pair<2>(u[x].y));
                        *reinterpret_cast<uint4*>(p + (to ^ 16)) =
                            make_uint4(kv8_pair<0>(u[x].z), kv8_pair<2>(u[x].z), kv8_pair<0>(u[x].w), kv8_pair<2>(u[x].w));
                    }
                }
                fence_proxy_async_shared();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sm.kv_full[buf]);
                    mbar_arrive(&sm.raw_empty[st]);
                }
                if (++st == F::RAW) st = 0, ph ^= 1;
            }
        }
    } else if (warp >= 4 && warp < 4 + 4 * F::NQ) {          // ---- softmax: a thread a row
        const int qi = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t s_addr = tmem + S_COL + 128 * qi + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t o_addr = tmem + O_COL + D * qi + ((uint32_t)((warp & 3) * 32) << 16);
        uint32_t s_ph = 0, o_ph = 0, g = 0, skipped = 0;
        bool ok = true, have = false;
        const float NONE = kv8_none();
        // of the piece at hand
        float m = NONE, l = 0.f;
        float own[2] = {0.f, 0.f};                           // l and n once they are apart
        int near = 0;
        bool whole = false, live = false;
        T* out = nullptr;
        float* part = nullptr;
        int64_t at_lse = 0;
        while (true) {
            Piece w;
            bool more;
            skipped = 0;
            while ((more = next_piece(w)) && w.rows - w.tile * ROWS <= 128 * qi) skipped += w.run;   // no rows for this group
            int power = 0;
            if (more) power = load_queries<T, D>(a, sm, w, qi, warp & 3, lane);
            if (have) {
                // ---- a row's result, or its part of one
                if (!kv8_wait(&sm.o_full[qi], o_ph, abort_flag, true)) break;
                o_ph ^= 1;
                tc_fence_after();
                const int pr = qi * 128 + row;
                float n = m - (near >> 2);
                if (near & 3) l = own[0], n = own[1];
                if (whole) {
                    store_row<T, D>(o_addr, live, kv8_inverse(m, n, l), out);
                    if (live && a.lse) a.lse[at_lse] = kv8_lse(n, l);
                } else {
                    store_row<float, D>(o_addr, live, 1.f, part + 3 * ROWS + (size_t)pr * D);
                    if (live) part[pr] = m, part[ROWS + pr] = l, part[2 * ROWS + pr] = n;
                }
                tc_fence_before();
            }
            if (!more) break;
            have = true;
            g += skipped;
            const int r = w.tile * ROWS + qi * 128 + row;
            live = r < w.rows;
            const int pos = w.len - w.n + (live ? r : w.tile * ROWS) / a.G;
            const int row_hi = a.causal ? min(w.len, pos + 1) : w.len;
            const int row_lo = a.window ? max(pos - a.window + 1, 0) : 0;
            const float qa = power == NO_NUMBERS ? -1.f : fabsf(a.scale) * __uint_as_float((uint32_t)(127 - power) << 23);
            whole = w.whole;
            out = static_cast<T*>(a.out) + kv8_out_row(a, w.q0, w.head, live ? r : 0, &at_lse);
            part = parts + ((size_t)cta * 2 + w.part) * kv8_part_floats(ROWS, D);
            m = NONE;
            l = 0.f;
            // tokens [safe_lo, safe_hi) are seen by all of the warp's rows
            const int safe_hi = __reduce_min_sync(0xffffffffu, live ? row_hi : 0x7fffffff);
            const int safe_lo = __reduce_max_sync(0xffffffffu, live ? row_lo : 0);

            for (int i = 0; i < w.run; ++i, ++g) {
                const int base = (w.first + i) * KT, slot = g & (CONS - 1);
                // (scores that are there mean that the slot's phase is this tile's)
                if (!kv8_wait(&sm.s_full[qi], s_ph, abort_flag, true) ||
                    !kv8_wait(&sm.cons_full[slot], g / CONS & 1, abort_flag, true)) {
                    ok = false;
                    break;
                }
                s_ph ^= 1;
                tc_fence_after();
                const float4* cons = sm.cons[slot];
                near = sm.near[slot];
                const bool inside = base >= safe_lo && base + KT <= safe_hi;
                const int lo = row_lo - base, hi = row_hi - base;
                const float t = inside ? tile_top(s_addr, cons, qa) : tile_top_some(s_addr, cons, qa, lo, hi);
                const bool raise = t > m + RAISE;
                if (__builtin_expect(__any_sync(0xffffffffu, raise || near & 3), 0)) {
                    if (__builtin_expect(near & 3, 0)) {
                        float sum = near & 1 ? l : own[0], n = near & 1 ? m - (near >> 2) : own[1];
                        tile_sum(s_addr, cons, qa, inside, sum, n);
                        own[0] = sum, own[1] = n;            // (l is of no use from here on)
                        tile_poison(s_addr, cons, inside);
                    }
                    const float now = raise ? t - HEAD : m;
                    const float f = raise ? exp2_fast(m - now) : 1.f;
                    m = now;
                    l *= f;
                    if (i > 0) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(o_addr + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            tmem_st_32x32b_x16(o_addr + 16 * c, o);
                        }
                    }
                }
                const float ref = m == NONE ? 0.f : m;
                l = inside ? tile_weights<F::TWO>(s_addr, cons, qa, ref, l) : tile_weights_some<F::TWO>(s_addr, cons, ref, l);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[qi]);
            }
            if (!ok) break;
            if (qa < 0.f) {                                  // (a row of zeros, of no numbers)
                if (l != 0.f) l = __int_as_float(0x7fffffff);
                if (own[0] != 0.f) own[0] = __int_as_float(0x7fffffff);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, 512);
}

// One CTA a SM, and none that could never have a tile.
int grid_of(const Kv8Attention& a) {
    const double rows = (double)a.c.T * a.G;
    const double most = (rows / 128 + a.c.seqs) * a.c.H * ((((int64_t)a.c.width << a.c.logB) + KT - 1) / KT);
    const int full = kv8_sm_count();
    return most < full ? (int)most : full;
}

template <class T, int D>
cudaError_t run(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    constexpr int ROWS = Form<T, D>::ROWS;
    static_assert(sizeof(Shared<T, D>) <= 232448, "shared memory of a CTA");
    cudaError_t e = cudaFuncSetAttribute(kv8_umma_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(Shared<T, D>));
    if (e != cudaSuccess) return e;
    const int grid = grid_of(a);
    float* parts = static_cast<float*>(scratch);
    Kv8Joint* joints = reinterpret_cast<Kv8Joint*>(parts + (size_t)grid * 2 * kv8_part_floats(ROWS, D));
    g_launched.store(true, std::memory_order_release);
    e = launch_pdl(kv8_umma_kernel<T, D>, dim3(grid), dim3(THREADS), sizeof(Shared<T, D>), st, a, parts, joints);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv8_join_kernel<T, D, ROWS, 1>, dim3(grid, ROWS / 32), dim3(KV8_JOIN_WARPS * 32), 0, st, a, (const float*)parts,
                      (const Kv8Joint*)joints);
}

template <class T>
cudaError_t run_d(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    return a.c.D == 64 ? run<T, 64>(a, scratch, st) : run<T, 128>(a, scratch, st);
}

}  // namespace

size_t kv8_umma_scratch(const Kv8Attention& a) {
    const int rows = a.dtype == TQ2_F32 ? 128 : 256;
    return (size_t)grid_of(a) * (2 * kv8_part_floats(rows, a.c.D) * sizeof(float) + sizeof(Kv8Joint));
}

cudaError_t launch_kv8_umma(const Kv8Attention& a, void* scratch, cudaStream_t st) {
    if (a.dtype == TQ2_F32) return run_d<float>(a, scratch, st);
    if (a.dtype == TQ2_F16) return run_d<__half>(a, scratch, st);
    return run_d<__nv_bfloat16>(a, scratch, st);
}

unsigned int read_clear_dev_error_kv8_umma(cudaStream_t st) { return read_clear_record(st); }

}  // namespace tq2
