// moe_stages.cuh -- shapes of the tcgen05 kernel of the routed experts, and the
// stage that each of its roles is at.  The roles walk the same stages by
// themselves, so all of them must see every change of the rings alike.
#pragma once

#include <cstdint>

namespace tq2 {

// Decoder groups (of four warps), epilogue warps and the columns one of those takes
// at a time.  Narrow tiles, whose MMAs are short, need three groups to feed them; the
// epilogue of wide ones, which the next tile's MMAs wait for, needs sixteen warps
// (64 experts of 2048x1024 bf16, top 8, 2048 tokens: 219 us with 2 groups and 16
// warps, 227 with 2 and 12, 230 with 3 and 12, 248 with 3 and 8).
template <bool WIDE>
struct MuShape {
    static constexpr int GROUPS = WIDE ? 2 : 3;
    static constexpr int HALF = WIDE ? 1 : 2;              // chunks of 64 k in half a stage
    static constexpr int STAGES = WIDE ? 4 : 3;            // stages of weights in tensor memory
    static constexpr int BN = WIDE ? 384 : 128;            // positions of a tile at most
    static constexpr int ACOL = WIDE ? 256 : 128;          // first tensor-memory column of the stages
    static constexpr int BLOCK_STAGES = 2 / HALF;          // stages of a packed block
    static constexpr int SLOTS = WIDE ? 5 : 4;             // activation slots (half a stage) of 32 KB
    static __host__ __device__ constexpr int raw(int G) { return WIDE ? 3 : G == 32 ? 4 : 5; }   // packed blocks of 256 k in their ring
    static constexpr int EPI = 4 + 4 * GROUPS;             // first epilogue warp
    static constexpr int DRAIN = WIDE ? 16 : 8;            // epilogue warps
    static constexpr int THREADS = 32 * (EPI + DRAIN);
    static constexpr int CW = 16;
};

// The stage at hand and the parities of its barriers' phases.  A tile of more
// than 256 (320) positions has its last accumulator columns where stage 0 (and
// 1) would be, so it goes without; a later tile that takes such a stage up again
// waits for `drained`, which the MMA warp completes then.  (Two groups of
// decoders need two stages: a group's last wait must be past every older phase
// of the stage that it waits for next.)
template <bool WIDE>
struct MuStages {
    int s = 0;
    int lowest = 0;                        // (stays 0 unless WIDE)
    uint32_t used = 0;
    // The next tile; returns how many stages it takes up again (negative: goes without).  Callers go by
    // this value alone: `lowest` has changed when it is there, so an expression must not hold both.
    __device__ __forceinline__ int begin(int cnt) {
        if (!WIDE) return 0;
        const int was = lowest;
        lowest = cnt > 320 ? 2 : cnt > 256 ? 1 : 0;
        s = s < lowest ? lowest : s;
        return was - lowest;
    }
    __device__ __forceinline__ void next() {
        used ^= 1u << s;
        s = s + 1 == MuShape<WIDE>::STAGES ? (WIDE ? lowest : 0) : s + 1;
    }
    __device__ __forceinline__ uint32_t parity() const { return (used >> s) & 1u; }
    // Activation slots (half a stage) in the ring, and their bytes.
    __device__ __forceinline__ int slots() const { return WIDE ? MuShape<WIDE>::SLOTS - lowest : MuShape<WIDE>::SLOTS; }
    __device__ __forceinline__ uint32_t slot_bytes() const { return WIDE ? 32768u + 8192u * (uint32_t)lowest : 32768u; }
};

}  // namespace tq2
