// moe_umma.cu -- the routed experts' products for many tokens, on tcgen05.
//
// Per matrix e of the plan, rows p of its positions, W = (c - z) d:
//   hidden[p] = silu(Gate x[p]) * (Up x[p]),   y[slot(p)] = Down hidden[p]
//
// Both products are D[n, p] = sum_k W[n,k] act[p,k] with 128 weight rows and up to
// 128 (wide tiles: 384) positions a tile, f16 operands and one f32 accumulator in
// tensor memory, in stages of 256 (128) k (what a stage costs besides its MMAs --
// waits, commits, hand-offs, several hundred cycles -- does not grow with its k):
//   * warps 0 and 2 stream the activations (B, 128-byte swizzle) by TMA, the first
//     and the second half of a stage (one warp takes ~650 cycles a slot);
//   * warp 3 streams the packed blocks of 256 k by bulk copies; narrow tiles are a
//     stream of weights, so they have five blocks (86 KB) in flight, wide ones three;
//   * two or three groups of four decoder warps, which take every second or third
//     stage, decode a block's rows, one weight row a thread, and store them as the A
//     operand in tensor memory (rounding (c - z) d to f16 is the only rounding of
//     the weights);
//   * warp 1 issues the MMAs; one barrier a stage covers both operands, and the
//     next stage's is tested while this stage's MMAs run;
//   * eight or sixteen epilogue warps drain the finished tile, some columns each in
//     turn, while the next tile's operands fill their rings.
// A matrix's weights are decoded once for each of its tiles, so wide tiles are as
// wide as tensor memory allows: 256 columns of accumulator leave room for four stages
// of weights, 320 for three, 384 for two.  (With 256 at most, experts of 257 rows were
// two tiles, each bound by the decoders: 2048 tokens of 64 experts 243 us against 219.)
// Bound: wide tiles by their MMAs (60 % of the time), the decoders and the epilogue,
// which nothing overlaps; narrow ones by the decoders (of 256 k in ~2200 cycles a
// group) and the blocks' latency: 213 MB of weights in 68 us from 40 to 64 tokens.
// Plan and first packed blocks are read while the kernel ahead ends (74 us without).
// A tile of the first product holds 64 rows of Gate and the same 64 of Up: lanes
// 0..15 of each quarter are Gate's, 16..31 Up's, so one shuffle meets the two.
//
// f16 holds the activations because each row is scaled by a power of two: a
// row of x so that its largest magnitude is 2^14..2^15, a hidden row by its
// bound |x|^2 bound(Gate) bound(Up) (Cauchy-Schwarz; silu(v) <= |v|), which
// can only be too large, for ordinary rows by about 2 D, and keeps every bit of
// values down to 2^-28 of it.  Where the rows of a matrix differ so much that its
// smallest might fall below, hidden rows are written in f32 and scaled by their own
// maximum in a pass of their own (own_scale; the rule and its cost are in q4_api.cu).
//
// silu goes by the fast exponential and division: off by a few 2^-22 of a value (times
// |v| for the exponential), far below the f16 that it is rounded to; v below -87, whose
// silu is next to nothing, may give 0.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/tq2.h"
#include "moe_stages.cuh"
#include "q4.cuh"
#include "tq2_internal.h"

namespace tq2 {

namespace {

constexpr int MU_A = 4;                    // stages of decoded weights at most
constexpr int MU_RAW = 5;                  // packed blocks of 256 k in their ring at most
constexpr int MU_LIST = 64;                // tiles of a CTA that are looked up ahead

// Activation rows in boxes of 32, 64, 128 and 256 (at most three copies a slot of
// a wide tile), or of 32, 64, 96 and 128 (one copy a chunk of a narrow one).
struct MuMaps {
    CUtensorMap box[4];
};

struct MuTile {
    int e, p0, cnt, r;
};

struct MuBars {
    uint64_t full[MU_A], empty[MU_A], half_empty[MU_A], raw_full[MU_RAW], raw_empty[MU_RAW];
    uint64_t acc_full, acc_empty, drained, idle;
    uint32_t tmem_base;
    int abort;
    MuTile list[MU_LIST];
    float2 scale[384];                     // epilogue: a tile's scales (or output rows and scales)
};

// Slot and phase parity of a ring's next item.
template <int S>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    bool first = true;                     // no slot has been used twice yet
    __device__ __forceinline__ void next() {
        if (++s == S) {
            s = 0;
            ph ^= 1u;
            first = false;
        }
    }
};

struct MuArgs {
    const uint8_t* w0;
    const uint8_t* w1;                     // pair: Up
    int64_t mstride;
    int nkc, zeros, E, nslots;
    int N;                                 // output columns (F, or D)
    int row_tiles;                         // tiles along them
    int K;
    int nk;                                // slots (half stages) of a tile
    int bn;                                // positions of a tile at most
    const int* offsets;
    const int* slots;
    const float2* scales;                  // [position] of a row of x: 1/scale; of the hidden row: scale
    void* hidden;                          // pair: [position][N], f16 or (own_scale) f32
    int own_scale;
    float* y;                              // else: [slot][N]
};

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]) : "memory");
}

__device__ __forceinline__ void put_hidden(float* p, float v) { *p = v; }
__device__ __forceinline__ void put_hidden(__half* p, float v) { *p = __float2half_rn(v); }

// Barrier of the epilogue warps.
template <int WARPS>
__device__ __forceinline__ void epi_bar() { asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory"); }

template <int G, bool PAIR, bool WIDE>
__global__ void __launch_bounds__(MuShape<WIDE>::THREADS, 1)
moe_umma_kernel(const __grid_constant__ MuMaps maps, const __grid_constant__ MuArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    constexpr int NG = Q4_K / G;
    constexpr int HALF = MuShape<WIDE>::HALF, ACOL = MuShape<WIDE>::ACOL, BLOCK_STAGES = MuShape<WIDE>::BLOCK_STAGES;
    constexpr int MU_GROUPS = MuShape<WIDE>::GROUPS, MU_EPI = MuShape<WIDE>::EPI, MU_THREADS = MuShape<WIDE>::THREADS;
    constexpr int CW = MuShape<WIDE>::CW, DRAIN = MuShape<WIDE>::DRAIN;
    constexpr int STEP = CW * DRAIN / 4;                   // columns that the epilogue warps of a quarter take in turn
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int blk = q4_block_bytes(G, a.zeros != 0);
    constexpr int RAW = MuShape<WIDE>::raw(G);
    uint8_t* raw_ring = smem + MuShape<WIDE>::SLOTS * 32768;
    MuBars* bars = reinterpret_cast<MuBars*>(raw_ring + RAW * 8 * blk);
    int* prefix = reinterpret_cast<int*>(bars + 1);        // token tiles before each matrix
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < MU_A; ++s) {
            mbar_init(&bars->full[s], 6);                  // two TMA producers and the stage's 4 decoder warps
            mbar_init(&bars->empty[s], 1);                 // the MMA warp's commits: a stage, its first 64 k
            mbar_init(&bars->half_empty[s], 1);
        }
        for (int r = 0; r < RAW; ++r) {
            mbar_init(&bars->raw_full[r], 1);
            mbar_init(&bars->raw_empty[r], 4 * BLOCK_STAGES);   // the decoder warps of its stages
        }
        mbar_init(&bars->acc_full, 1);
        mbar_init(&bars->acc_empty, DRAIN);                    // every epilogue warp
        mbar_init(&bars->drained, 1);                      // the MMA warp
        mbar_init(&bars->idle, 1);                         // its last commit
        bars->abort = 0;
        fence_mbar_init();
        for (int i = 0; i < 4; ++i) tma_prefetch_desc(&maps.box[i]);
    }
    if (warp == 2) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    pdl_launch_dependents();
    if (warp == 1) {
        // The plan is there: the kernel ahead lets this one start only when it has waited for it, and so for the
        // first packed blocks; what that kernel writes is waited for below.
        int run = 0;
        bool down = false;                                 // ranges that go back are no plan: nothing is done
        for (int e0 = 0; e0 <= a.E; e0 += 32) {
            const int e = e0 + lane;
            const int o = e <= a.E ? plan_offset(a.offsets, a.nslots, e) : 0;
            const int rows = e < a.E ? plan_offset(a.offsets, a.nslots, e + 1) - o : 0;
            const int n = (rows + a.bn - 1) / a.bn;
            down |= rows < 0;
            int s = n;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += up;
            }
            if (e <= a.E) prefix[e] = run + s - n;
            run += __shfl_sync(0xffffffffu, s, 31);
        }
        __syncwarp();
        if (__any_sync(0xffffffffu, down) && lane == 0) prefix[a.E] = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort;
    const int total = prefix[a.E] * a.row_tiles;

    // tile t: row tiles fastest; a matrix's positions are cut evenly
    auto find_tile = [&](int t) {
        MuTile m;
        const int tt = t / a.row_tiles;
        m.r = t - tt * a.row_tiles;
        int lo = 0, hi = a.E;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= tt) lo = mid; else hi = mid;
        }
        m.e = lo;
        const int i = tt - prefix[lo], n = prefix[lo + 1] - prefix[lo], o = plan_offset(a.offsets, a.nslots, lo),
                  c = plan_offset(a.offsets, a.nslots, lo + 1) - o;
        const int each = c / n, more = c - each * n;
        m.p0 = o + i * each + min(i, more);
        m.cnt = each + (i < more ? 1 : 0);
        return m;
    };
    // this CTA's i-th tile
    const int mine = total > (int)blockIdx.x ? (total - blockIdx.x - 1) / gridDim.x + 1 : 0;
    for (int i = tid; i < min(mine, MU_LIST); i += MU_THREADS) bars->list[i] = find_tile(blockIdx.x + i * gridDim.x);
    __syncthreads();
    auto tile_at = [&](int i) { return i < MU_LIST ? bars->list[i] : find_tile(blockIdx.x + i * gridDim.x); };
    const int stages = (a.nk + 1) / 2;                     // the last one maybe a half

    if (warp == 0 || warp == 2) {                          // ---- activations
        pdl_wait();
        if (elect_one()) {
            // The ring's slots are cut anew where a tile has another number of them than the one before: after
            // that one's last MMA, while its accumulator is drained.  Otherwise slot n is free after the MMAs
            // of slot n - slots, whose stage `old` follows `late` stages behind.
            const int half = warp >> 1;                    // first or second 64 k of the stages
            MuStages<WIDE> f, old;
            bool ok = true;
            int slot = half, run = 0;                      // stages since the ring was cut
            uint32_t armed = 0, parity = 0;                // stages whose full barrier was armed, and for which phase
            uint64_t* last = nullptr;                      // of the stage before
            uint32_t last_parity = 0;
            for (int i = 0; i < mine && ok; ++i) {
                const MuTile m = tile_at(i);
                const int boxes = (m.cnt + 31) / 32;
                if (f.begin(m.cnt) != 0) {
                    if (last && !mbar_wait_or_abort(last, last_parity, abort_flag)) {
                        ok = false;
                        break;
                    }
                    slot = half;
                    run = 0;
                }
                if (run == 0) old = f;
                const int slots = f.slots();
                const uint32_t bytes = f.slot_bytes();
                // slot 2 st + half - slots
                const int late = (slots - half + 1) / 2;
                uint64_t* freed = (slots - half) & 1 ? bars->empty : bars->half_empty;
                for (int st = 0; st < stages; ++st) {
                    if (run >= late) {
                        if (!mbar_wait_or_abort(&freed[old.s], old.parity(), abort_flag)) {
                            ok = false;
                            break;
                        }
                        old.next();
                    }
                    ++run;
                    const bool there = 2 * st + half < a.nk;   // the last stage may be one slot
                    uint64_t* bar = &bars->full[f.s];
                    armed |= 1u << f.s;
                    parity = (parity & ~(1u << f.s)) | f.parity() << f.s;
                    mbar_arrive_expect_tx(bar, there ? (uint32_t)boxes * (4096u * HALF) : 0u);
                    if (there) {
                        uint8_t* dst = smem + (uint32_t)slot * bytes;
                        const int k0 = (2 * st + half) * (64 * HALF);
                        if (WIDE) {
                            int row = m.p0;
#pragma unroll
                            for (int x = 3; x >= 0; --x)
                                if (boxes & (1 << x)) {
                                    tma_load_2d(dst, &maps.box[x], bar, k0, row);
                                    dst += 4096 << x;
                                    row += 32 << x;
                                }
                        } else {                           // (a chunk past the row's end is zeros)
                            tma_load_2d(dst, &maps.box[boxes - 1], bar, k0, m.p0);
                            tma_load_2d(dst + boxes * 4096, &maps.box[boxes - 1], bar, k0 + 64, m.p0);
                        }
                    }
                    slot += 2;
                    slot -= slot >= slots ? slots : 0;
                    last = &bars->empty[f.s];
                    last_parity = f.parity();
                    f.next();
                }
            }
            // After a wait that ran out the copies already issued must land before the CTA exits.  Each is
            // short of its barrier's phase, which may never complete: give them their (bounded) time.
            if (!ok) {
                *abort_flag = 1;
                for (int x = 0; x < MU_A; ++x)
                    if ((armed >> x) & 1u) mbar_wait(&bars->full[x], (parity >> x) & 1u);
            }
        }
        __syncwarp();
    } else if (warp == 3) {
        if (elect_one()) {                                 // ---- packed blocks
            Ring<RAW> r;
            bool ok = true;
            const uint32_t bytes = 8u * (uint32_t)blk;
            for (int i = 0; i < mine && ok; ++i) {
                const MuTile m = tile_at(i);
                // first of the tile's blocks of a chunk: 8 row tiles of one matrix, or 4 of each of two
                const int rt = PAIR ? m.r * 4 : m.r * 8;
                const int64_t first = (int64_t)m.e * a.mstride + q4_block_index(rt, 0, a.nkc) * blk;
                for (int kc = 0; kc < a.nkc; ++kc, r.next()) {
                    if (!r.first && !mbar_wait_or_abort(&bars->raw_empty[r.s], r.ph ^ 1u, abort_flag)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&bars->raw_full[r.s], bytes);
                    uint8_t* dst = raw_ring + (size_t)r.s * bytes;
                    const int64_t at = first + (int64_t)kc * 8 * blk;
                    if (PAIR) {
                        bulk_load(dst, a.w0 + at, bytes / 2, &bars->raw_full[r.s]);
                        bulk_load(dst + bytes / 2, a.w1 + at, bytes / 2, &bars->raw_full[r.s]);
                    } else {
                        bulk_load(dst, a.w0 + at, bytes, &bars->raw_full[r.s]);
                    }
                }
            }
            if (!ok)
                for (int i = 0; i < RAW; ++i)
                    mbar_wait(&bars->raw_full[i], i < r.s ? r.ph : r.ph ^ 1u);
        }
    } else if (warp == 1) {                                // ---- MMA issuer
        if (elect_one()) {
            int slot = 0;                                  // of the stage's first 64 k
            MuStages<WIDE> f;
            bool ok = true;
            int cnt = mine > 0 ? tile_at(0).cnt : 0;
            for (int i = 0; i < mine && ok; ++i) {
                // more than 256 positions are two MMAs side by side
                const int n16 = (cnt + 15) / 16 * 16, n1 = WIDE && cnt > 256 ? (n16 / 16 + 1) / 2 * 16 : n16, n2 = n16 - n1;
                const int boxes = (cnt + 31) / 32;
                const uint32_t idesc = idesc_f16_f32(128, (uint32_t)n1), idesc2 = idesc_f16_f32(128, (uint32_t)n2);
                if (i > 0) {
                    if (!mbar_wait_or_abort(&bars->acc_empty, (uint32_t)(i - 1) & 1u, abort_flag, true)) {
                        *abort_flag = 1;
                        break;
                    }
                }
                const int again = f.begin(cnt);
                if (again > 0) mbar_arrive(&bars->drained);
                if (again != 0) slot = 0;
                const int slots = f.slots();
                const uint32_t bytes = f.slot_bytes();
                bool ready = false;
                tc_fence_after();
                for (int st = 0; st < stages; ++st) {
                    if (!ready && !mbar_wait_or_abort(&bars->full[f.s], f.parity(), abort_flag, true)) {
                        *abort_flag = 1;
                        ok = false;
                        break;
                    }
                    MuStages<WIDE> g = f;
                    g.next();
                    // (its latency hides under the MMAs below)
                    ready = st + 1 < stages && mbar_test_wait(&bars->full[g.s], g.parity());
                    tc_fence_after();
                    const uint32_t acol = tmem + ACOL + (uint32_t)(f.s * 64 * HALF);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (h == 0 || 2 * st + 1 < a.nk) {
                            const uint64_t bdesc = sdesc_kmajor_sw128(smem_u32(smem + (uint32_t)slot * bytes));
#pragma unroll
                            for (int c = 0; c < HALF; ++c)
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    umma_f16_ts(tmem, acol + (uint32_t)((h * HALF + c) * 32 + j * 8),
                                                bdesc + (uint64_t)(2 * j) + (uint64_t)(c * boxes * 256), idesc,
                                                (st > 0 || h > 0 || c > 0 || j > 0) ? 1u : 0u);
                            if (WIDE && n2) {
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    umma_f16_ts(tmem + (uint32_t)n1, acol + (uint32_t)(h * 32 + j * 8),
                                                bdesc + (uint64_t)(2 * j + n1 * 8), idesc2,
                                                (st > 0 || h > 0 || j > 0) ? 1u : 0u);
                            }
                        }
                        if (++slot == slots) slot = 0;
                        umma_commit(h == 0 ? &bars->half_empty[f.s] : &bars->empty[f.s]);
                    }
                    f = g;
                }
                if (!ok) break;
                umma_commit(&bars->acc_full);
                if (i + 1 < mine) cnt = tile_at(i + 1).cnt;
            }
            // Whatever the other roles gave up, the MMAs still in flight end before tensor memory is given back and
            // the CTA exits.  (Without a timeout the epilogue waits for the same ones.)
            umma_commit(&bars->idle);
            mbar_wait(&bars->idle, 0u);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < MU_EPI) {               // ---- decoders
        // quarter q of the rows, the group's stages of the CTA's sequence; rows 0..15 of a
        // quarter are one 16-row tile's, 16..31 the next one's (pair: Gate's and Up's)
        const int q = warp & 3;
        const int row = lane & 15, g = row & 7, hi = row >> 3;
        const int b = PAIR ? (lane >> 4) * 4 + q : q * 2 + (lane >> 4);
        const uint32_t expo = q4_exponent<false>();
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16) + ACOL;
        // The stage at hand: of tile i, `st` of its stages; its packed block is the CTA's item `item`, in slot rs.
        MuStages<WIDE> f;
        int i = 0, st = 0, base = 0, item = 0, rs = 0;
        uint32_t rph = 0, drains = 0;
        bool ok = true, owed = false;                      // owed: a wait for `drained`
        if (mine > 0) f.begin(tile_at(0).cnt);
        auto advance = [&] {                               // by one stage
            f.next();
            if (++st == stages) {
                st = 0;
                base += a.nkc;
                ++i;
                if (WIDE && i < mine) owed = f.begin(tile_at(i).cnt) > 0 || owed;
            }
        };
        auto settle = [&] {
            const int now = base + st / BLOCK_STAGES;
            rs += now - item;
            item = now;
            if (rs >= RAW) {                               // (an item or two were the other groups')
                rs -= RAW;
                rph ^= 1u;
            }
        };
        for (int x = (warp - 4) >> 2; x > 0; --x) advance();
        settle();
        while (i < mine) {
            // The stage first, then its packed block: the MMAs of its last use are past the slot's last block, so
            // that the parity waited for is the right one's.  (The first passes at a stage's first use.)
            if (owed) {
                ok = mbar_wait_or_abort(&bars->drained, drains & 1u, abort_flag);
                ++drains;
                owed = false;
            }
            if (!ok || !mbar_wait_or_abort(&bars->empty[f.s], f.parity() ^ 1u, abort_flag) ||
                !mbar_wait_or_abort(&bars->raw_full[rs], rph, abort_flag)) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after();
            const uint8_t* src = raw_ring + (size_t)rs * 8 * blk + b * blk;
            const uint8_t* sc = src + Q4_CODES + q4_scale_index(row, 0, NG) * 2;
            const uint8_t* zp = src + Q4_CODES + 32 * NG + q4_scale_index(row, 0, NG);
            // (a last stage's missing second half is decoded from the block's padding and not used)
#pragma unroll
            for (int h = 0; h < HALF; ++h) {
                const int c0 = 2 * h + (BLOCK_STAGES == 2 ? 2 * (st & 1) : 0);   // two chunks of 64 k
                uint2 w[2][4];
#pragma unroll
                for (int at = 0; at < 2; ++at)
#pragma unroll
                    for (int tt = 0; tt < 4; ++tt)
                        w[at][tt] = *reinterpret_cast<const uint2*>(src + (c0 + at) * 512 + (tt * 8 + g) * 16 + hi * 8);
#pragma unroll
                for (int at = 0; at < 2; ++at) {
                    const int c = c0 + at;
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        uint32_t v[16];
                        const int gi = (c * 2 + half) / (G / 32);
                        const __half2 d = __half2half2(*reinterpret_cast<const __half*>(sc + gi * 4));
                        const Q4Zero z = q4_zero<false>(a.zeros ? zp[gi * 2] : 8u);
#pragma unroll
                        for (int tt = 0; tt < 4; ++tt) {
                            uint32_t p[4];
                            q4_decode<false>(half ? w[at][tt].y : w[at][tt].x, expo, z, p);
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                const __half2 m = __hmul2(*reinterpret_cast<const __half2*>(&p[x]), d);
                                v[4 * tt + x] = *reinterpret_cast<const uint32_t*>(&m);
                            }
                        }
                        tmem_st_32x32b_x16(lane_addr + (uint32_t)(f.s * 64 * HALF + (2 * h + at) * 32 + 16 * half), v);
                    }
                }
            }
            tmem_wait_st();
            tc_fence_before();
            // the packed values are used: the slot is refilled through the async proxy
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&bars->full[f.s]);
                mbar_arrive(&bars->raw_empty[rs]);
                // (a last block of one stage has one group)
                if (BLOCK_STAGES == 2 && (stages & 1) && st == stages - 1) mbar_arrive(&bars->raw_empty[rs]);
            }
#pragma unroll
            for (int x = 0; x < MU_GROUPS; ++x) advance();
            settle();
        }
    } else if (warp >= MU_EPI) {                           // ---- epilogue: CW columns in turn
        const int q = warp & 3, b = (warp - MU_EPI) >> 2;
        const uint32_t lane_addr = tmem + ((uint32_t)(q * 32) << 16);
        pdl_wait();
        bool ok = true;
        for (int ti = 0; ti < mine; ++ti) {
            const MuTile m = tile_at(ti);
            epi_bar<DRAIN>();                                     // the last tile's scales and rows are done with
            for (int i = tid - MU_EPI * 32; i < m.cnt; i += DRAIN * 32) {
                float2 sc = a.scales[m.p0 + i];
                if (!PAIR) sc.x = __int_as_float(plan_slot(a.slots, a.nslots, m.p0 + i));
                bars->scale[i] = sc;
            }
            epi_bar<DRAIN>();
            // (after a wait that ran out a warp stays for the barriers: others may still be on their way to them)
            if (!ok || !mbar_wait_or_abort(&bars->acc_full, (uint32_t)ti & 1u, abort_flag)) {
                *abort_flag = 1;
                ok = false;
                continue;
            }
            tc_fence_after();
            // pair: this lane finishes half of CW positions of its row, else all of them
            const bool upper = PAIR && lane >= 16;
            const int n = PAIR ? m.r * 64 + q * 16 + (lane & 15) : m.r * 128 + q * 32 + lane;
            const bool in = n < a.N;
            bool held = true;
            uint32_t v[CW], w[CW];
            // the columns after the ones at hand are read ahead; with the last ones the accumulator is handed back
            auto read = [&](uint32_t (&x)[CW], int cc) {
                tmem_ld_32x32b_x16(lane_addr + (uint32_t)cc, x);
                tmem_wait_ld();
                if (cc + STEP >= m.cnt) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->acc_empty);
                    held = false;
                }
            };
            auto finish = [&](const uint32_t (&x)[CW], int cc) {
                if (PAIR) {
                    constexpr int H = CW / 2;
                    const int c0 = cc + (upper ? H : 0), left = in ? m.cnt - c0 : 0;
                    const int64_t at = (int64_t)(m.p0 + c0) * a.N + n;
                    auto store = [&](auto* out, bool scaled) {
#pragma unroll
                        for (int i = 0; i < H; ++i, out += a.N) {
                            const uint32_t other = __shfl_xor_sync(0xffffffffu, upper ? x[i] : x[H + i], 16);
                            const float2 sc = bars->scale[c0 + i];
                            const float gt = __uint_as_float(upper ? other : x[i]) * sc.x;
                            const float up = __uint_as_float(upper ? x[H + i] : other) * sc.x;
                            const float hv = __fdividef(gt, 1.0f + __expf(-gt)) * up;
                            if (i < left) put_hidden(out, scaled ? hv * sc.y : hv);
                        }
                    };
                    if (a.own_scale) store(static_cast<float*>(a.hidden) + at, false);
                    else store(static_cast<__half*>(a.hidden) + at, true);
                } else if (in) {
                    float* out = a.y + n;
                    const int left = m.cnt - cc;
                    auto put = [&](int i) {
                        const float2 sc = bars->scale[cc + i];
                        out[(int64_t)__float_as_int(sc.x) * a.N] = __uint_as_float(x[i]) * sc.y;
                    };
                    if (left >= CW) {
#pragma unroll
                        for (int i = 0; i < CW; ++i) put(i);
                    } else {
#pragma unroll
                        for (int i = 0; i < CW; ++i)
                            if (i < left) put(i);
                    }
                }
            };
            if (CW * b < m.cnt) read(v, CW * b);
            for (int cc = CW * b; cc < m.cnt; cc += 2 * STEP) {
                if (cc + STEP < m.cnt) read(w, cc + STEP);
                finish(v, cc);
                if (cc + STEP < m.cnt) {
                    if (cc + 2 * STEP < m.cnt) read(v, cc + 2 * STEP);
                    finish(w, cc + STEP);
                }
            }
            if (held) {                                    // a narrow tile: no columns for this warp
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->acc_empty);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Pairs of f16 or bf16.
template <class T>
struct Pair;
template <>
struct Pair<__half> {
    using type = __half2;
    static __device__ __forceinline__ float2 f32(__half2 v) { return __half22float2(v); }
    static __device__ __forceinline__ __half2 zero() { return __float2half2_rn(0.f); }
};
template <>
struct Pair<__nv_bfloat16> {
    using type = __nv_bfloat162;
    static __device__ __forceinline__ float2 f32(__nv_bfloat162 v) { return __bfloat1622float2(v); }
    static __device__ __forceinline__ __nv_bfloat162 zero() { return __float2bfloat162_rn(0.f); }
};
// Eight elements of a row.
template <class T>
__device__ __forceinline__ void load8(const T* p, bool vec, typename Pair<T>::type (&v)[4]) {
    if (vec) {
        *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    } else {
        T raw[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) raw[i] = p[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i].x = raw[2 * i];
            v[i].y = raw[2 * i + 1];
        }
    }
}

// Of each routed slot: its position and the product of its matrices' bounds.
__global__ void __launch_bounds__(256)
moe_where_kernel(const int* __restrict__ offsets, const int* __restrict__ slots, int nslots, int E,
                 const float* __restrict__ bound0, const float* __restrict__ bound1, float2* __restrict__ where) {
    pdl_launch_dependents();
    pdl_wait();
    const int p = blockIdx.x * 256 + threadIdx.x;
    if (p >= plan_offset(offsets, nslots, E)) return;
    int lo = 0, hi = E;                                    // the position's matrix
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (plan_offset(offsets, nslots, mid) <= p) lo = mid; else hi = mid;
    }
    where[plan_slot(slots, nslots, p)] = make_float2(__int_as_float(p), bound0[lo] * bound1[lo]);
}

// Exponent bits of the power of two that takes a row of largest magnitude m to 2^14..2^15, kept a
// normal number with a normal inverse; 1 for a row of zeros or one with infinities.
__device__ __forceinline__ int scale_exponent(float m) {
    const int be = (__float_as_int(m) >> 23) & 255;
    const int se = be == 0 ? 253 : 127 + 14 - (be - 127);
    return m == 0.f || be == 255 ? 127 : min(se, 253);
}

// A CTA a token: its row of x as f16, scaled, at each of its positions, and the
// scales.  A row is converted once for all its positions (a warp a position took 745
// instructions for each: 21 us for 16384 slots of 2048, now 15; the whole call of 2048
// tokens of 64 experts 227 -> 221); what is left is bound by the writes of T*k*D halves.
template <class T>
__global__ void __launch_bounds__(256)
moe_stage_kernel(const T* __restrict__ x, int64_t ldx, int vec, int D, const int* __restrict__ ids,
                 const float2* __restrict__ where, int nslots, int k, __half* __restrict__ xs,
                 float2* __restrict__ first, float2* __restrict__ second) {
    __shared__ int to[32];                                 // positions, -1: none
    __shared__ float red[9];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_launch_dependents();                               // (the products read the plan before they wait)
    const int64_t t = blockIdx.x;
    const T* row = x + t * ldx;
    typename Pair<T>::type v[4], top[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = top[i] = Pair<T>::zero();
    float2 at = make_float2(0.f, 0.f);
    int pos = -1;
    if (tid < k && ids[t * k + tid] >= 0) {
        at = where[t * k + tid];
        pos = min(max(__float_as_int(at.x), 0), nslots - 1);
    }
    for (int c = tid * 8; c < D; c += 2048) {
        load8(row + c, vec != 0, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = __hmax2(top[i], __habs2(v[i]));
    }
    top[0] = __hmax2(__hmax2(top[0], top[1]), __hmax2(top[2], top[3]));
    float m = fmaxf(Pair<T>::f32(top[0]).x, Pair<T>::f32(top[0]).y);
    m = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(m)));   // m >= 0: its bits have its order
    if (lane == 0) red[warp] = m;
    if (tid < 32) to[tid] = pos;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    const int se = scale_exponent(m);
    const float s = __int_as_float(se << 23);
    float ss = 0.f;
    for (int c = tid * 8; c < D; c += 2048) {
        if (D > 2048) load8(row + c, vec != 0, v);         // (else they are at hand)
        __half2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f = Pair<T>::f32(v[i]);
            f.x *= s;
            f.y *= s;
            ss = fmaf(f.x, f.x, ss);
            ss = fmaf(f.y, f.y, ss);
            h[i] = __float22half2_rn(f);
        }
#pragma unroll 4
        for (int j = 0; j < k; ++j) {
            const int p = to[j];
            if (p >= 0) *reinterpret_cast<uint4*>(xs + (int64_t)p * D + c) = *reinterpret_cast<uint4*>(h);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    __syncthreads();
    if (lane == 0) red[warp] = ss;
    __syncthreads();
    if (pos >= 0) {
        ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += red[i];
        // exponent of the hidden row's bound, x's own scale taken out
        const float b = ss * at.y;
        const int e = ((__float_as_int(b) >> 23) & 255) - 127 - 2 * (se - 127);
        int hs = 127 + 14 - e;
        if (b == 0.f) hs = 127;
        hs = hs < 1 ? 1 : hs > 253 ? 253 : hs;
        const float inv = __int_as_float((254 - se) << 23);
        first[pos] = make_float2(inv, __int_as_float(hs << 23));
        second[pos] = make_float2(0.f, __int_as_float((254 - hs) << 23));
    }
}

// A CTA a position: its f32 gated row as f16, scaled by its own maximum, and the
// scale for the second product.  (That product reads the plan before it waits, so it may
// start only when this kernel has waited.)
__global__ void __launch_bounds__(256)
moe_rescale_kernel(const float* __restrict__ rows, const int* __restrict__ offsets, int nslots, int E, int F,
                   __half* __restrict__ out, float2* __restrict__ second) {
    __shared__ float red[8];
    const int tid = threadIdx.x, p = blockIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (p >= plan_offset(offsets, nslots, E)) return;
    const float4* row = reinterpret_cast<const float4*>(rows + (int64_t)p * F);
    float m = 0.f;
    for (int c = tid; c < F / 4; c += 256) {
        const float4 v = row[c];
        m = fmaxf(fmaxf(fmaxf(m, fabsf(v.x)), fmaxf(fabsf(v.y), fabsf(v.z))), fabsf(v.w));
    }
    m = __int_as_float(__reduce_max_sync(0xffffffffu, __float_as_int(m)));
    if ((tid & 31) == 0) red[tid >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, red[i]);
    const int se = scale_exponent(m);
    const float s = __int_as_float(se << 23);
    for (int c = tid; c < F / 4; c += 256) {
        const float4 v = row[c];
        const __half2 h[2] = {__floats2half2_rn(v.x * s, v.y * s), __floats2half2_rn(v.z * s, v.w * s)};
        reinterpret_cast<uint2*>(out + (int64_t)p * F)[c] = *reinterpret_cast<const uint2*>(h);
    }
    if (tid == 0) second[p] = make_float2(0.f, __int_as_float((254 - se) << 23));
}

template <int G, bool PAIR, bool WIDE>
cudaError_t launch_umma_moe(const MuMaps& maps, MuArgs a, cudaStream_t st) {
    // more than 256 positions to a tile need a store of every decoder group in each tile (four stages)
    a.nk = (a.K + 64 * MuShape<WIDE>::HALF - 1) / (64 * MuShape<WIDE>::HALF);
    a.bn = WIDE && a.nk <= 6 ? 256 : MuShape<WIDE>::BN;
    int dev = 0, sms = 152;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const size_t smem = 1024 + (size_t)MuShape<WIDE>::SLOTS * 32768 + (size_t)MuShape<WIDE>::raw(G) * 8 * q4_block_bytes(G, a.zeros != 0) +
                        sizeof(MuBars) + (size_t)(a.E + 1) * 4;
    cudaError_t e = cudaFuncSetAttribute(moe_umma_kernel<G, PAIR, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_umma_kernel<G, PAIR, WIDE>, dim3((unsigned)sms), dim3(MuShape<WIDE>::THREADS), smem, st,
                      maps, a);
}

// f16 rows of length `inner`.
bool row_maps(MuMaps& m, __half* rows, int64_t inner, int64_t n, bool wide) {
    for (int i = 0; i < 4; ++i)
        if (!make_tensor_map_2d(&m.box[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rows, (uint64_t)inner, (uint64_t)n,
                                (uint64_t)inner * 2, 64u, wide ? 32u << i : 32u * (i + 1), CU_TENSOR_MAP_SWIZZLE_128B))
            return false;
    return true;
}

// Wide tiles from 112 rows a matrix on average (64 experts of 2048x1024, 112 / 128
// rows each: narrow 122 / 141 us, wide 121 / 127; the one shape that was measured).  (Two groups of decoders need
// blocks of two stages: a slot's last block must have been theirs or the MMAs'.)
bool wide_tiles(int64_t nslots, int64_t E, int64_t K) { return nslots >= 112 * E && K > 128; }

template <bool PAIR>
cudaError_t launch_by_group(int group, __half* rows, const MuArgs& a, cudaStream_t st) {
    const bool wide = wide_tiles(a.nslots, a.E, a.K);
    MuMaps maps;
    if (!row_maps(maps, rows, a.K, a.nslots, wide)) return cudaErrorInvalidValue;
    if (group == 32)
        return wide ? launch_umma_moe<32, PAIR, true>(maps, a, st) : launch_umma_moe<32, PAIR, false>(maps, a, st);
    if (group == 64)
        return wide ? launch_umma_moe<64, PAIR, true>(maps, a, st) : launch_umma_moe<64, PAIR, false>(maps, a, st);
    return wide ? launch_umma_moe<128, PAIR, true>(maps, a, st) : launch_umma_moe<128, PAIR, false>(maps, a, st);
}

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

// f16 rows of x and of the hidden values and two pairs of scales by position; a position and a bound by slot;
// the hidden values in f32 where they are scaled afterwards.
size_t moe_tensor_scratch(int64_t nslots, int64_t D, int64_t F, bool own_scale) {
    return round256((size_t)nslots * D * 2) + round256((size_t)nslots * F * 2) + 3 * round256((size_t)nslots * 8) +
           (own_scale ? (size_t)nslots * F * 4 : 0);
}

cudaError_t launch_moe_tensor(const MoeTensor& m, void* scratch, cudaStream_t st) {
    g_launched.store(true, std::memory_order_release);
    const int64_t S = m.nslots, D = m.gate->K, F = m.gate->N;
    char* at = static_cast<char*>(scratch);
    __half* xs = reinterpret_cast<__half*>(at);
    at += round256((size_t)S * D * 2);
    __half* hid = reinterpret_cast<__half*>(at);
    at += round256((size_t)S * F * 2);
    float2* first = reinterpret_cast<float2*>(at);
    at += round256((size_t)S * 8);
    float2* second = reinterpret_cast<float2*>(at);
    at += round256((size_t)S * 8);
    float2* where = reinterpret_cast<float2*>(at);
    at += round256((size_t)S * 8);
    float* hid32 = reinterpret_cast<float*>(at);
    const int E = (int)m.gate->E;
    const unsigned T = (unsigned)(S / m.k);
    const int vec = (reinterpret_cast<uintptr_t>(m.x) & 15) == 0 && m.ldx % 8 == 0;
    cudaError_t e = launch_pdl(moe_where_kernel, dim3((unsigned)((S + 255) / 256)), dim3(256), 0, st, m.offsets,
                               m.slots, (int)S, E, static_cast<const float*>(m.gate->bound),
                               static_cast<const float*>(m.up->bound), where);
    if (e != cudaSuccess) return e;
    if (m.dtype == TQ2_F16)
        e = launch_pdl(moe_stage_kernel<__half>, dim3(T), dim3(256), 0, st, static_cast<const __half*>(m.x), m.ldx,
                       vec, (int)D, m.ids, static_cast<const float2*>(where), (int)S, m.k, xs, first, second);
    else
        e = launch_pdl(moe_stage_kernel<__nv_bfloat16>, dim3(T), dim3(256), 0, st,
                       static_cast<const __nv_bfloat16*>(m.x), m.ldx, vec, (int)D, m.ids,
                       static_cast<const float2*>(where), (int)S, m.k, xs, first, second);
    if (e != cudaSuccess) return e;
    MuArgs a{};
    a.w0 = m.gate->blocks;
    a.w1 = m.up->blocks;
    a.mstride = m.gate->mstride;
    a.nkc = (int)m.gate->nkc;
    a.zeros = m.gate->zeros ? 1 : 0;
    a.E = E;
    a.nslots = (int)S;
    a.N = (int)F;
    a.row_tiles = (int)((F + 63) / 64);
    a.K = (int)D;
    a.offsets = m.offsets;
    a.slots = m.slots;
    a.scales = first;
    a.hidden = m.own_scale ? static_cast<void*>(hid32) : hid;
    a.own_scale = m.own_scale ? 1 : 0;
    e = launch_by_group<true>(m.gate->group, xs, a, st);
    if (e == cudaSuccess && m.own_scale)
        e = launch_pdl(moe_rescale_kernel, dim3((unsigned)S), dim3(256), 0, st, static_cast<const float*>(hid32),
                       m.offsets, (int)S, E, (int)F, hid, second);
    if (e != cudaSuccess) return e;
    MuArgs b = a;
    b.w0 = m.down->blocks;
    b.w1 = nullptr;
    b.mstride = m.down->mstride;
    b.nkc = (int)m.down->nkc;
    b.zeros = m.down->zeros ? 1 : 0;
    b.N = (int)D;
    b.row_tiles = (int)((D + 127) / 128);
    b.K = (int)F;
    b.scales = second;
    b.hidden = nullptr;
    b.y = m.y;
    return launch_by_group<false>(m.down->group, hid, b, st);
}

unsigned int read_clear_dev_error_moe_umma(cudaStream_t st) { return read_clear_record(st); }

}  // namespace tq2
