// moe_rows.h -- dispatch's rows as the experts' products take them: whose row is whose, tiles of one expert's rows, fetches
// into LDS, and the activation behind the sums (gfx950, wave64).
#ifndef MOE_ROWS_H
#define MOE_ROWS_H

#include "moe_types.h"

namespace moe_detail {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));      // loads and stores at less than their size's alignment
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));

struct Tile {
    int expert, row, end;                  // rows row..end-1 of the expert, whose last row is end - 1
};

// Where each expert's rows and row tiles begin: expert e's rows follow expert e-1's, and each expert starts a tile of
// its own. One copy in each workgroup's LDS, made once: workgroups stay for many tiles.
struct Plan {
    uint32_t row[kMaxExperts + 1], tile[kMaxExperts + 1];
    uint32_t part[2][8];
    int expert;
};

// Fills the plan for tiles of BM rows and returns their number. The counts are ep_recv_count's differences, held
// within [0, rows] whatever the array holds. All threads call it. (Args: erc, ep_recv_count; W, epr, E; S segments of a
// rank; rows.)
template <int BM, int THREADS, class Args>
__device__ int make_plan(const Args &a, Plan &plan)
{
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    constexpr int kEach = kMaxExperts / THREADS;
    const uint32_t most = (uint32_t)a.rows;
    uint32_t count[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int e = tid * kEach + i;
        count[i] = 0;
        if (e < a.E) {
            const int r = e / a.epr, el = e - r * a.epr;
            const int32_t *p = a.erc + (size_t)r * a.S + (size_t)(el + 1) * a.W - 1;
            const int cur = min(max(p[0], 0), a.rows), prev = el ? min(max(p[-a.W], 0), a.rows) : 0;
            count[i] = (uint32_t)max(cur - prev, 0);
        }
        sum = min(most, sum + count[i]);
    }
    // rows before this thread's experts
    uint32_t inc = wave_scan(sum, most);
    if (lane == kWave - 1) plan.part[0][wave] = inc;
    uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)inc, 0x138, 0xf, 0xf, false);    // one lane up
    __syncthreads();
    for (int i = 0; i < wave; ++i) before = min(most, before + plan.part[0][i]);
    uint32_t start[kEach + 1], tiles = 0;
    start[0] = before;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        start[i + 1] = min(most, start[i] + count[i]);
        tiles += (start[i + 1] - start[i] + BM - 1) / BM;
    }
    inc = wave_scan(tiles, 0x7fffffffu);
    if (lane == kWave - 1) plan.part[1][wave] = inc;
    uint32_t at = inc - tiles;
    __syncthreads();
    for (int i = 0; i < wave; ++i) at += plan.part[1][i];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        plan.row[tid * kEach + i] = start[i];
        plan.tile[tid * kEach + i] = at;
        at += (start[i + 1] - start[i] + BM - 1) / BM;
    }
    if (tid == THREADS - 1) {
        plan.row[kMaxExperts] = start[kEach];
        plan.tile[kMaxExperts] = at;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(plan.tile[kMaxExperts]);
}

// Row tile `mt` of the plan (below its number of tiles). All threads call it; it holds a barrier.
template <int BM, int THREADS, class Args>
__device__ Tile find_tile(const Args &a, Plan &plan, int mt)
{
    for (int e = threadIdx.x; e < a.E; e += THREADS)
        if (plan.tile[e] <= (uint32_t)mt && (uint32_t)mt < plan.tile[e + 1]) plan.expert = e;
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(plan.expert);
    return Tile{e, (int)__builtin_amdgcn_readfirstlane(plan.row[e] + (mt - plan.tile[e]) * BM),
                (int)__builtin_amdgcn_readfirstlane(plan.row[e + 1])};
}

// silu(gate) * up by the hardware's exponential and reciprocal (an ulp each; the exponent's argument is off by |gate|
// half steps): far below the 16-bit rounding behind it. Below a gate of about -87 the reciprocal underflows, where fp32's
// exponential overflows below -88, and the result is 0 instead of less than 2e-36 |up|.
__device__ __forceinline__ float swiglu(float gate, float up)
{
    return gate * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(gate * -1.44269504f)) * up;
}

// A buffer of `bytes` from `base` on (the same in all lanes); reads past it give zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *base, uint64_t bytes)
{
    const int size = (int)(bytes < 0xffffffffull ? (uint32_t)bytes : 0xffffffffu);
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(base), 0, size, 0x00027000);
}
// 16 bytes a lane from `buffer`, `lane` + `all` bytes in, to LDS, the wavefront's 1 KiB one after the other from `to`,
// past the registers. (A buffer load: the compiler takes a global load of this kind for one that may count as an LDS
// access too, and then waits for every LDS read at the first.)
__device__ __forceinline__ void fetch_lds(__amdgpu_buffer_rsrc_t buffer, uint32_t lane, uint32_t all, u32x4 *to)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (__attribute__((address_space(3))) void *)to, 16, (int)lane, (int)all,
                                             0, 0);
}
// A barrier behind which every wavefront's LDS reads and writes, and all but its youngest LEFT fetches into LDS, are
// done. (The wait is the builtin: the compiler then knows which fetches are in and puts no wait of its own before the
// reads. The fence of __syncthreads would wait for all of them; the empty asm keeps memory accesses in their place.)
template <int LEFT>
__device__ __forceinline__ void barrier_fetched()
{
    static_assert(LEFT < 64, "vmcnt has 6 bits");
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0070 | (LEFT & 15) | (LEFT >> 4) << 14);      // vmcnt LEFT, lgkmcnt 0
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace moe_detail

#endif  // MOE_ROWS_H
