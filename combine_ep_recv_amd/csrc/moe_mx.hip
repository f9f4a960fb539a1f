// moe_mx.hip -- microscaled rows and the experts' product on them (gfx950, wave64).
//
// OCP Microscaling (MX v1.0): 32 consecutive elements of a row share one power of two, stored as an E8M0 byte
// (2^(byte - 127)); elements are E2M1 (4 bits, two a byte, the even one in the low nibble) or E4M3 (8 bits).
//   quantise    shared = clamp(floor(log2 max|x|) - emax, -127, 127), code = nearest of x * 2^-shared, ties to even
//   dequantise  code * 2^shared
//   product     out[row] = act(sum_k x[row, k] * w[e(row), n, k]), both sides microscaled, the weights E2M1; row
//               `row` belongs to expert e(row) by ep_recv_count; summed in fp32, rounded once.

#include "moe_types.h"

#include <limits.h>

#include <algorithm>
#include <type_traits>

namespace {

using namespace moe_detail;

constexpr int kBlock = 32;                 // elements that share a scale byte
constexpr int kPiece = 16;                 // elements a lane quantises: half a block
constexpr int kMxThreads = 256;
constexpr long long kMaxBlocks = (1ll << 31) - kMxThreads / 2;      // two lanes a block: a launch has below 2^32 lanes

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));      // loads and stores at less than their size's alignment
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a8 __attribute__((aligned(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// --------------------------------------------------------------------------
// quantise and dequantise
// --------------------------------------------------------------------------

struct MxArgs {
    const void *in;
    void *out;
    const uint8_t *scales_in;
    uint8_t *scales_out;
    long long pieces;          // 16-element pieces in all
    int per_row, blocks;       // pieces and blocks of a row
};

constexpr long long kOnceBytes = 256ll << 20;      // the Infinity Cache

// 16 elements of T (16-byte aligned: a row is a multiple of 16 elements)
template <class T, bool ONCE>
__device__ __forceinline__ void load_piece(const void *in, long long piece, float (&x)[kPiece])
{
    const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const typename T::raw *>(in) + piece * kPiece);
    if constexpr (sizeof(typename T::raw) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4 v = ONCE ? __builtin_nontemporal_load(p + i) : p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = __uint_as_float(v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 v = ONCE ? __builtin_nontemporal_load(p + i) : p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = T::load((uint16_t)(v[j] & 0xffff));
                x[8 * i + 2 * j + 1] = T::load((uint16_t)(v[j] >> 16));
            }
        }
    }
}

// A lane takes 16 elements and its neighbour the block's other half; a row with a last block of 16 leaves that
// block to one lane. E: MOE_MX_E2M1 or MOE_MX_E4M3. ONCE: the input passes the caches by.
//
// Memory bounds it: 2 bytes in and about half a byte (E2M1) or one (E4M3) out, an element, against some ten
// instructions. Loads of 32 bytes a lane are whole lines between neighbours, the shared exponent is one exchange of
// neighbours away, and nothing passes through LDS. bf16 [32768, 7168] to E2M1 and back to bf16 takes 204 us, 5.8 TB/s
// of its 1.19 GB (a large copy reaches 5.2); [256, 7168] is the two calls, 17 us, 6 of them
// on the card.
template <class T, int E, bool RAGGED, bool ONCE>
__global__ __launch_bounds__(kMxThreads) void quantize_kernel(MxArgs a)
{
    const uint32_t lane_piece = blockIdx.x * kMxThreads + threadIdx.x;
    // RAGGED: the grid counts two pieces for every block, and the half that a row's last block lacks is empty
    long long row = 0, piece = lane_piece;
    bool live;
    if (RAGGED) {
        const uint32_t r = lane_piece / (2u * a.blocks), q = lane_piece - r * (2u * a.blocks);
        row = r;
        piece = row * a.per_row + q;
        live = piece < a.pieces && q < (uint32_t)a.per_row;
    } else {
        live = piece < a.pieces;
    }
    float x[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = 0.f;
    if (live) load_piece<T, ONCE>(a.in, piece, x);
    // the largest magnitude as bits: ordered like the values, and infinity and NaN above them all
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < kPiece; ++i) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    constexpr int emax = E == MOE_MX_E2M1 ? 2 : 8;
    // floor(log2) of a normal binary32 is its exponent field - 127; a subnormal's is below -126, so that the byte
    // is 0 as for a zero block
    const int field = (int)(top >> 23);
    const bool finite = field < 255;
    const int byte = finite ? max(field - emax, 0) : 255;
    const float up = __uint_as_float((uint32_t)(254 - (finite ? byte : 254)) << 23);     // 2^(127 - byte), exact
    if (!live) return;
    if constexpr (E == MOE_MX_E2M1) {
        u32x2 code;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t c = 0;
            const float *v = x + 8 * h;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * up, v[1] * up, 1.f, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * up, v[3] * up, 1.f, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * up, v[5] * up, 1.f, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * up, v[7] * up, 1.f, 3);
            code[h] = finite ? c : 0;
        }
        reinterpret_cast<u32x2 *>(a.out)[piece] = code;
    } else {
        u32x4 code;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = fminf(fmaxf(x[4 * h + i] * up, -448.f), 448.f);
            int c = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
            c = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], c, true);
            code[h] = finite ? (uint32_t)c : 0;
        }
        reinterpret_cast<u32x4 *>(a.out)[piece] = code;
    }
    if (RAGGED) {
        const int q = (int)(piece - row * a.per_row);
        if (!(q & 1)) a.scales_out[row * a.blocks + q / 2] = (uint8_t)byte;
    } else if (!(piece & 1)) {
        a.scales_out[piece / 2] = (uint8_t)byte;
    }
}

// The operand that the scaled conversions take for a scale byte: they read the exponent field of a binary32 as the
// E8M0 byte, 0 (2^-127) and 255 (NaN) among them. (Multiplying afterwards would let the compiler fold the product
// into the fp16 conversion as a fused multiply-add to +0, which turns -0 into +0.)
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

template <class T, int E, bool RAGGED>
__global__ __launch_bounds__(kMxThreads) void dequantize_kernel(MxArgs a)
{
    const uint32_t lane_piece = blockIdx.x * kMxThreads + threadIdx.x;
    const long long piece = lane_piece;
    if (piece >= a.pieces) return;
    long long block = piece / 2;
    if (RAGGED) {
        const uint32_t row = lane_piece / (uint32_t)a.per_row;
        block = (long long)row * a.blocks + (lane_piece - row * a.per_row) / 2;
    }
    const float s = scale_of(a.scales_in[block]);
    float x[kPiece];
    if constexpr (E == MOE_MX_E2M1) {
        const u32x2 c = reinterpret_cast<const u32x2 *>(a.in)[piece];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const f32x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], s, 0);
            const f32x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], s, 1);
            const f32x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], s, 2);
            const f32x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c[h], s, 3);
            const f32x2 v[4] = {v0, v1, v2, v3};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[8 * h + 2 * i] = v[i][0];
                x[8 * h + 2 * i + 1] = v[i][1];
            }
        }
    } else {
        const u32x4 c = reinterpret_cast<const u32x4 *>(a.in)[piece];
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const f32x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[h], s, false);
            const f32x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(c[h], s, true);
            x[4 * h] = lo[0];
            x[4 * h + 1] = lo[1];
            x[4 * h + 2] = hi[0];
            x[4 * h + 3] = hi[1];
        }
    }
    u32x4 *out = reinterpret_cast<u32x4 *>(static_cast<typename T::raw *>(a.out) + piece * kPiece);
    if constexpr (sizeof(typename T::raw) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __float_as_uint(x[4 * i + j]);
            out[i] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = (uint32_t)T::store(x[8 * i + 2 * j]) | ((uint32_t)T::store(x[8 * i + 2 * j + 1]) << 16);
            out[i] = v;
        }
    }
}

// --------------------------------------------------------------------------
// the experts' product
// --------------------------------------------------------------------------

constexpr int kMaxExperts = 1024;          // dispatch's limits
constexpr int kMinWorld = 2, kMaxWorld = 768;
constexpr int kStep = 128;                 // elements of k in one matrix instruction
constexpr int kSuper = 4 * kStep;          // ... in a group of four, whose 16 scale bytes are one load
// At most as many workgroups as run at once, two of the small tiles on each of 256 CUs and one of the larger ones: they
// stay, and make the plan once. 64 experts, E2M1, 7168 -> 4096 with SwiGLU, 128 and 512 rows each: 292 and 651 us with
// 256, 296 and 663 with 512, 309 and 668 with 1024; small tiles, 512 -> 1024 over 256 experts with 32 rows each: 28.6,
// 24.6 and 27.0.
constexpr int kWorkgroupsSmall = 512, kWorkgroupsLarge = 256;

struct ProductArgs {
    const uint8_t *x, *xs, *w, *ws;
    const int32_t *erc;
    void *out;
    int W, epr, E, S, rows, k, n, nb, fo;  // nb: blocks of a row; fo: columns of out
    int ntiles;
};

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

// Inclusive sums over the 64 lanes that stop at `most` (which keeps them in 32 bits and in order; sums that never
// reach it are plain ones).
__device__ __forceinline__ uint32_t wave_scan(uint32_t v, uint32_t most)
{
#define MOE_SCAN_STEP(CTRL, ROWS) v = min(most, v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false));
    MOE_SCAN_STEP(0x111, 0xf)          // row shifts by 1, 2, 4 and 8
    MOE_SCAN_STEP(0x112, 0xf)
    MOE_SCAN_STEP(0x114, 0xf)
    MOE_SCAN_STEP(0x118, 0xf)
    MOE_SCAN_STEP(0x142, 0xa)          // the last lane of a row to the next row, of the lower half to the upper one
    MOE_SCAN_STEP(0x143, 0xc)
#undef MOE_SCAN_STEP
    return v;
}

// Fills the plan for tiles of BM rows and returns their number. The counts are ep_recv_count's differences, held
// within [0, rows] whatever the array holds. All threads call it.
template <int BM, int THREADS>
__device__ int make_plan(const ProductArgs &a, Plan &plan)
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
template <int BM, int THREADS>
__device__ Tile find_tile(const ProductArgs &a, Plan &plan, int mt)
{
    for (int e = threadIdx.x; e < a.E; e += THREADS)
        if (plan.tile[e] <= (uint32_t)mt && (uint32_t)mt < plan.tile[e + 1]) plan.expert = e;
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(plan.expert);
    return Tile{e, (int)__builtin_amdgcn_readfirstlane(plan.row[e] + (mt - plan.tile[e]) * BM),
                (int)__builtin_amdgcn_readfirstlane(plan.row[e + 1])};
}

// The instruction adds its 128 products in fp32 when both sides are E2M1 (a sum of whole numbers below 2^24 comes out
// exactly). With E4M3 it aligns neighbouring products to the largest of them and drops what lies more than 13 bits
// below it. E4M3 products span 20 bits, so that nothing right would be left where the large ones cancel. So E4M3 rows are
// multiplied in two parts (see split), each of which keeps every product; sums are fp32 throughout.
//
// One 16 x 16 x 128 step: weights (E2M1) by rows of elements of format XF (0: E4M3, 4: E2M1), the scale bytes in
// byte SEL of ws and xs. Lane (r, g), r = lane % 16, g = lane / 16, holds 32 elements of row r and the scale of
// its row's block g: E2M1 elements 32g..32g+31; E4M3 elements 16g..16g+15 and 64+16g..64+16g+15. Result register
// i is weight row 4g + i, input row r.
template <int XF, int SEL>
__device__ __forceinline__ f32x4 mma(i32x8 w, i32x8 x, f32x4 c, uint32_t ws, uint32_t xs)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, XF, SEL, (int)ws, SEL, (int)xs);
}

// E4M3 codes in two parts: the magnitudes from 2 on (whose code has bit 6 set) and those below, zeros in each other's
// places. The first are whole multiples of 2^-2 up to 448, the second of 2^-9 below 2: times E2M1 (multiples of 1/2 up
// to 6) a part's products span 13 bits below the largest possible one's power of two, which is what the instruction
// keeps. (A selector byte above 12 makes v_perm's byte 0xff, 0 picks a byte of the zeros.)
__device__ __forceinline__ void split(i32x8 x, i32x8 &upper, i32x8 &lower)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        upper[i] = x[i] & (int)__builtin_amdgcn_perm(0u, 0u, (uint32_t)x[i] & 0x40404040u);
        lower[i] = x[i] ^ upper[i];
    }
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi)
{
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// 16 bytes of a step, piece p of a row (`row` points at its own first piece), with zeros past the row's k elements
template <int XF>
__device__ __forceinline__ u32x4 load_piece_or_zero(const uint8_t *row, int at, int p, int k)
{
    constexpr int kElems = XF == 4 ? 32 : 16;
    const int first = at + p * kElems;
    u32x4 v = {0, 0, 0, 0};
    const uint8_t *q = row + (XF == 4 ? at / 2 : at);
    if (first + kElems <= k) v = *reinterpret_cast<const u32x4_a8 *>(q);
    else if (first < k) {                              // E2M1 only: half a block
        const u32x2 h = *reinterpret_cast<const u32x2 *>(q);
        v[0] = h[0];
        v[1] = h[1];
    }
    return v;
}
// The scale bytes of a row in four steps, 16 of them, as a word for each g: byte g of every word, a transpose of 4 x 4
// bytes.
__device__ __forceinline__ u32x4 by_group(u32x4 d)
{
    const uint32_t a = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), b = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u), e = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
    return u32x4{__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u),
                 __builtin_amdgcn_perm(e, c, 0x05040100u), __builtin_amdgcn_perm(e, c, 0x07060302u)};
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

// Rows of one expert, 16 * FR * WM at a time, against 16 * NF * WN weight rows (half of them the gate's, half the
// matching ones of the up projection with GLU): WM x WN wavefronts, each with FR x NF fragments of its own and all of k.
//
// Both sides go through LDS: a matrix instruction's lane holds 16 bytes of a row whose neighbours sit in lanes 16
// apart, so loading straight into its layout makes the cache look at every lane's 16 bytes by itself (one look-up a
// clock), where eight adjacent lanes that read a line of 128 bytes count as one. A stage is 128 bytes of an input
// row, kSub instruction steps: 256 elements of E2M1, 128 of E4M3. The 16-byte pieces of a row are swapped by its number
// (each lane fetches the piece that belongs where it writes) so that the eight lanes that LDS serves in a clock meet
// every bank once.
//
// LDS holds RING stages. The barrier comes when the current one has been read, two fragments before its end; behind it
// the stage RING ahead is fetched in its place, and the next one's first fragments are read while those two multiply.
// E4M3 fragments are parted one ahead.
// With two stages the next one is on its way while one is multiplied; with four, three are, for shapes that wait for
// the weights from device memory. Input fragments are read two ahead. Scale bytes come 512 elements (four steps) at a
// time, through registers, and become a word per (row, g) on the way. (Two groups at a time, so that neighbouring lanes
// share a request: 1161 us for 1181 with many rows, but 23.0 for 21.7 with two tokens, whose code is then read once.)
//
// What bounds it, with 64 experts of 7168 -> 4096 with SwiGLU or 256 of 2048 -> 7168. Few rows: the weights' bytes,
// 212 us for 1.0 GB with 32 rows of E2M1 each (a plain read reaches 6.2 TB/s), 234 with E4M3, whose two parts
// take twice the matrix instructions and 32 others a fragment, and 505 us for 2.4 GB in and out with 96 rows each. Many
// E4M3 rows: 1505 us with 512 rows each, where the matrix instructions alone take 860 at the nominal clock; it falls to
// 1.9 GHz, of whose cycles the matrix units are busy in 59 %. Many E2M1 rows,
// skewed (1024 a rank, 8 ranks): 1110 us or 3.5 PFLOP/s, where the same instructions alone on random values reach 7.1 and on
// constant ones 8.4. Power takes the clock from 2.4 GHz to 1.6 or 1.7; of those cycles the matrix units are busy in 52 % and
// LDS reads in 28 %, and wavefronts wait for 41 % of their time, an eighth of that for LDS. Cut down (from 1150 us): 840
// without fetches and results, 930 without fetches, 1070 with fetches that hit the cache: the loop's own waits cost more
// than memory. Four wavefronts of 128 x 128, which read a third less from LDS, need 1300: one wavefront a SIMD leaves its
// waits open.
template <class T, int XF, int FR, int NF, int WM, int WN, int SUB, int RING, bool GLU>
__global__ __launch_bounds__(WM *WN *kWave, 2) void expert_product_kernel(ProductArgs a)
{
    constexpr int kThreads = WM * WN * kWave, kRowsW = WN * NF * 16, kRowsX = WM * FR * 16;
    constexpr int kSub = XF == 4 ? SUB : 1, kStages = 4 / kSub;   // steps of a stage, stages of 512 elements
    constexpr int kPw = 4 * kSub, kPx = XF == 4 ? kPw : 8;    // 16-byte pieces of a row in a stage
    constexpr int kLoadsW = kRowsW * kPw / kThreads, kLoadsX = kRowsX * kPx / kThreads, kLoads = kLoadsW + kLoadsX;
    // Whether a wavefront multiplies only the fragments that hold rows of the expert. E4M3's two parts make a fragment
    // dear: 64 experts of 64 rows, 7168 -> 4096 with SwiGLU, 303 us, 380 with every fragment; two tokens 22 and 41.
    constexpr bool kSkip = XF != 4;
    static_assert(!kSkip || FR == 4, "the counts of fragments that the main loop is made for");
    constexpr int kRows = kRowsW + kRowsX, kScales = (kRows + kThreads - 1) / kThreads;   // scale rows of a thread
    static_assert(kRowsW * kPw % kThreads == 0 && kRowsX * kPx % kThreads == 0, "every thread carries as many pieces");
    static_assert(RING == 2 || (RING == 4 && kStages == 4), "a stage's place in the ring is known where it is used");
    // a stage's weights, then its inputs; an array a stage, so that the compiler tells them apart
    constexpr int kSizeW = kRowsW * kPw, kSize = kSizeW + kRowsX * kPx;
    __shared__ u32x4 l0[kSize], l1[kSize], l2[RING == 4 ? kSize : 1], l3[RING == 4 ? kSize : 1];
    __shared__ u32x4 s0[kRows], s1[kRows];
    auto ring = [&](int i) -> u32x4 * { return i % RING == 0 ? l0 : (i % RING == 1 ? l1 : (i % RING == 2 ? l2 : l3)); };
    __shared__ Plan plan;
    const int total = make_plan<kRowsX, kThreads>(a, plan) * a.ntiles;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), wm = wave / WN, wn = wave % WN;
    const int r = lane % 16, g = lane / 16;
    constexpr int kOut = GLU ? NF / 2 : NF, kOwn = NF * 16;   // output fragments and weight rows of a wavefront
    const int half = a.n / 2;
    const uint32_t wrow = a.k / 2, xrow = XF == 4 ? a.k / 2 : a.k;
    const int supers = a.k / kSuper, stages = supers * kStages;
    // piece p of row q in LDS, for rows of 4 and of 8 pieces
    auto place4 = [](int q, int p) { return q * 4 + (p ^ ((q >> 1) & 3)); };
    auto place8 = [](int q, int p) { return q * 8 + (p ^ (q & 7)); };
    // a reader's pieces: of fragment 0, the others lie 16 rows apart
    const int lo = place8(r, g), hi = place8(r, 4 + g);
    const int wfrag[2] = {wn * kOwn * kPw + (kPw == 8 ? lo : place4(r, g)), wn * kOwn * kPw + hi};
    const int xfrag[2] = {wm * FR * 16 * kPx + (kPx == 8 ? lo : place4(r, g)), wm * FR * 16 * kPx + hi};
    // the piece that this thread fetches of its rows (rows of its later pieces are a multiple of 8 on)
    const int p8 = tid % 8 ^ (tid / 8 % 8), p4 = tid % 4 ^ (tid / 8 % 4);
    const int pw = kPw == 8 ? p8 : p4, px = kPx == 8 ? p8 : p4;

    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const Tile tile = find_tile<kRowsX, kThreads>(a, plan, t / a.ntiles);
        const int tile0 = t % a.ntiles * (WN * kOut * 16);
        const uint8_t *wb = a.w + (size_t)tile.expert * a.n * wrow, *wsb = a.ws + (size_t)tile.expert * a.n * a.nb;
        const uint8_t *xb = a.x + (size_t)tile.row * xrow, *xsb = a.xs + (size_t)tile.row * a.nb;
        const __amdgpu_buffer_rsrc_t wbuf = buffer_of(wb, (uint64_t)a.n * wrow);
        const __amdgpu_buffer_rsrc_t xbuf = buffer_of(xb, (uint64_t)(tile.end - tile.row) * xrow);
        const int last = tile.end - 1 - tile.row;             // rows past the expert's last read the last one
        // weight row of a place in the tile; columns past the last one read the last one's, and are not stored
        auto weight_row = [&](int q) -> uint32_t {
            const int c = GLU ? q / kOwn * (kOwn / 2) + q % (kOwn / 2) : q;
            return (GLU && q % kOwn >= kOwn / 2 ? half : 0) + min(tile0 + c, a.fo - 1);
        };
        uint32_t wo[kLoadsW], xo[kLoadsX];
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) wo[i] = weight_row((tid + i * kThreads) / kPw) * wrow + 16 * pw;
#pragma unroll
        for (int i = 0; i < kLoadsX; ++i) xo[i] = (uint32_t)min((tid + i * kThreads) / kPx, last) * xrow + 16 * px;
        // scale rows: the weights', then the inputs'; threads past the last one carry it too (the same bytes)
        const uint8_t *sp[kScales];
        int sq[kScales];
#pragma unroll
        for (int i = 0; i < kScales; ++i) {
            sq[i] = min(tid + i * kThreads, kRows - 1);
            sp[i] = sq[i] < kRowsW ? wsb + (size_t)weight_row(sq[i]) * a.nb : xsb + (size_t)min(sq[i] - kRowsW, last) * a.nb;
        }

        f32x4 acc[FR][NF];
#pragma unroll
        for (int f = 0; f < FR; ++f)
#pragma unroll
            for (int j = 0; j < NF; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};

        u32x4 raw[kScales];
        // Fetches of whole stages. Beyond the last one the last one is fetched again, and not used: a branch here would
        // part the steps that it stands between, and the waits count the fetches.
        auto fetch = [&](int stage, int slot) {
            const uint32_t at = min(stage, stages - 1);
            u32x4 *wl = ring(slot), *xl = wl + kSizeW;
#pragma unroll
            for (int i = 0; i < kLoadsW; ++i) fetch_lds(wbuf, wo[i], at * (16 * kPw), wl + i * kThreads + wave * kWave);
#pragma unroll
            for (int i = 0; i < kLoadsX; ++i) fetch_lds(xbuf, xo[i], at * (16 * kPx), xl + i * kThreads + wave * kWave);
        };
        auto load_scales = [&](int super) {
            const uint32_t at = min(super, supers - 1) * 16;
#pragma unroll
            for (int i = 0; i < kScales; ++i) raw[i] = *reinterpret_cast<const u32x4_a1 *>(sp[i] + at);
        };
        auto keep_scales = [&](u32x4 *to) {
#pragma unroll
            for (int i = 0; i < kScales; ++i) to[sq[i]] = by_group(raw[i]);
        };
        i32x8 wf[2][NF], xf[FR], upper[2], lower[2];
        uint32_t ws[NF], xs[FR];
        // fragments of step i of 512 elements
        auto read_w = [&](int i) {
            const u32x4 *l = ring(i / kSub) + wfrag[i % kSub];
#pragma unroll
            for (int j = 0; j < NF; ++j) wf[i & 1][j] = join(l[j * 16 * kPw], l[j * 16 * kPw]);
        };
        auto read_x = [&](int i, int f) {
            const u32x4 *l = ring(i / kSub) + kSizeW + f * 16 * kPx;
            xf[f] = XF == 4 ? join(l[xfrag[i % kSub]], l[xfrag[i % kSub]]) : join(l[xfrag[0]], l[xfrag[1]]);
        };
        // E4M3: the parts of fragment f, made while the one before multiplies
        auto part = [&](int f) {
            if constexpr (XF != 4) split(xf[f], upper[f & 1], lower[f & 1]);
        };
        auto multiply = [&](auto step, int f) {
            constexpr int I = decltype(step)::value;
#pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[f][j] = mma<XF, I>(wf[I & 1][j], XF == 4 ? xf[f] : upper[f & 1], acc[f][j], ws[j], xs[f]);
            if (XF != 4) {
#pragma unroll
                for (int j = 0; j < NF; ++j)
                    acc[f][j] = mma<XF, I>(wf[I & 1][j], lower[f & 1], acc[f][j], ws[j], xs[f]);
            }
        };
        auto read_scales = [&](const u32x4 *from) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(from) + g;
#pragma unroll
            for (int j = 0; j < NF; ++j) ws[j] = p[(wn * kOwn + j * 16 + r) * 4];
#pragma unroll
            for (int f = 0; f < FR; ++f) xs[f] = p[(kRowsW + (wm * FR + f) * 16 + r) * 4];
        };
        // Whole groups of 512 elements, for the wavefront's first LIVE fragments. Every wavefront meets the same barriers
        // and makes the same fetches whatever its LIVE.
        auto whole = [&](auto count) {
            constexpr int LIVE = decltype(count)::value, LAST = LIVE < 2 ? LIVE : 2;
            load_scales(0);
#pragma unroll
            for (int i = 0; i < RING - 1; ++i) fetch(i, i);
            __builtin_amdgcn_sched_barrier(0);
            keep_scales(s0);
            barrier_fetched<(RING - 2) * kLoads>();
            fetch(RING - 1, RING - 1);
            read_w(0);
#pragma unroll
            for (int f = 0; f < LAST; ++f) read_x(0, f);
            read_scales(s0);
            part(0);
            for (int super = 0; super < supers; ++super) {
#define MOE_WIDE_STEP(I)                                                                              \
                {                                                                                     \
                    constexpr bool kEnd = I % kSub == kSub - 1;                                       \
                    if (I == 0) load_scales(super + 1);                                               \
                    if (I == 3) keep_scales(s1);                                                      \
                    _Pragma("unroll") for (int f = 0; f < LIVE - LAST; ++f) {                         \
                        read_x(I, f + 2);                                                             \
                        multiply(std::integral_constant<int, I>(), f);                                \
                        if (f + 1 < LIVE - 1) part(f + 1);                                            \
                        __builtin_amdgcn_sched_barrier(0);                                            \
                    }                                                                                 \
                    if (LIVE > 1) part(LIVE - 1);                                                     \
                    if (kEnd) {                                                                       \
                        barrier_fetched<(RING - 2) * kLoads>();                                       \
                        __builtin_amdgcn_sched_barrier(0);                                            \
                        fetch(super * kStages + I / kSub + RING, I / kSub);                           \
                        __builtin_amdgcn_sched_barrier(0);                                            \
                    }                                                                                 \
                    read_w((I + 1) & 3);                                                              \
                    _Pragma("unroll") for (int f = 0; f < LAST; ++f) read_x((I + 1) & 3, f);          \
                    __builtin_amdgcn_sched_barrier(0);                                                \
                    _Pragma("unroll") for (int f = LIVE - LAST; f < LIVE; ++f)                        \
                        multiply(std::integral_constant<int, I>(), f);                                \
                    part(0);                                                                          \
                    if (I == 3) read_scales(s1);                                                      \
                    __builtin_amdgcn_sched_barrier(0);                                                \
                }
                MOE_WIDE_STEP(0)
                MOE_WIDE_STEP(1)
                MOE_WIDE_STEP(2)
                MOE_WIDE_STEP(3)
#undef MOE_WIDE_STEP
            }
        };
        if (supers > 0) {
            using std::integral_constant;
            if constexpr (kSkip) {
                const int live = (last + 16 - wm * FR * 16) / 16;      // fragments of this wavefront that hold rows
                if (live > 3) whole(integral_constant<int, 4>());
                else if (live == 3) whole(integral_constant<int, 3>());
                else if (live == 2) whole(integral_constant<int, 2>());
                else whole(integral_constant<int, 1>());
            } else {
                whole(integral_constant<int, FR>());
            }
        }
        barrier_fetched<0>();
        // the last k % 512 elements, a step at a time
        for (int at = supers * kSuper; at < a.k; at += kStep) {
            constexpr int kTx = XF == 4 ? 4 : 8;              // pieces of an input row in one step
#pragma unroll 1
            for (int c = tid; c < kRowsW * 4; c += kThreads)
                l0[kPw == 8 ? place8(c / 4, c % 4) : place4(c / 4, c % 4)] =
                    load_piece_or_zero<4>(wb + weight_row(c / 4) * wrow + 16 * (c % 4), at, c % 4, a.k);
#pragma unroll 1
            for (int c = tid; c < kRowsX * kTx; c += kThreads)
                l0[kSizeW + (kPx == 8 ? place8(c / kTx, c % kTx) : place4(c / kTx, c % kTx))] =
                    load_piece_or_zero<XF>(xb + (uint32_t)min(c / kTx, last) * xrow + 16 * (c % kTx), at, c % kTx, a.k);
            const int b = at / kBlock;
#pragma unroll
            for (int j = 0; j < kScales; ++j) {
                u32x4 v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = b + i < a.nb ? sp[j][b + i] : 127;
                s0[sq[j]] = v;
            }
            __syncthreads();
            read_w(0);
            read_scales(s0);
#pragma unroll
            for (int f = 0; f < FR; ++f) {
                read_x(0, f);
                part(f);
                multiply(std::integral_constant<int, 0>(), f);
            }
            __syncthreads();
        }
        // Results leave by way of LDS, 16 rows of the wavefront's columns at a time, so that neighbouring lanes store
        // neighbouring 16 bytes: a lane's own four columns are 8 bytes 16 lanes from the next ones, each a look-up of
        // its own in the cache. (16 ranks of 256 tokens,
        // 2048 -> 7168: 530 us, 560 with 8-byte stores; 515 since the stores pass the cache by.)
        constexpr int kPitch = kOut * 32 + 16;                // bytes; 16 more than the columns, to spread the banks
        constexpr int kLanes = kOut * 2;                      // lanes of a row
        char *own = reinterpret_cast<char *>(l0) + wave * 16 * kPitch;
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            wave_fence();
#pragma unroll
            for (int j = 0; j < kOut; ++j) {
                f32x4 v = acc[f][j];
                if (GLU) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], acc[f][j + kOut][i]);
                }
                u32x2 u;
                u[0] = (uint32_t)T::store(v[0]) | ((uint32_t)T::store(v[1]) << 16);
                u[1] = (uint32_t)T::store(v[2]) | ((uint32_t)T::store(v[3]) << 16);
                *reinterpret_cast<u32x2 *>(own + r * kPitch + j * 32 + g * 8) = u;
            }
            wave_fence();
#pragma unroll
            for (int i = 0; i < kOut * 32; i += kWave) {      // pieces of 16 bytes
                const int q = i + lane, row = tile.row + (wm * FR + f) * 16 + q / kLanes;
                const int col = tile0 + wn * kOut * 16 + q % kLanes * 8;
                if (q / kLanes >= 16 || row >= tile.end || col >= a.fo) continue;
                const u32x4 v = *reinterpret_cast<const u32x4 *>(own + q / kLanes * kPitch + q % kLanes * 16);
                typename T::raw *out = static_cast<typename T::raw *>(a.out) + (size_t)row * a.fo + col;
                if (col + 8 <= a.fo) {
                    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_a2 *>(out));
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (col + c < a.fo) out[c] = (typename T::raw)(v[c / 2] >> (c % 2 * 16));
                }
            }
        }
    }
}

// Rows of a tile, for `each` rows an expert (masked pairs' among them: no more is known here). A tile of 64 rows keeps
// three stages of weights on their way and pads few rows; above 48 rows an expert it would read the weights a second
// time, through the cache, and do too little on what it read. Measured with 64 experts, 7168 -> 4096 with SwiGLU, 32 / 48
// / 64 rows each: E4M3 233 / 275 / 348 us with 64 rows, 277 / 292 / 302 with 128; E2M1 218 / 247 / 288 and 212 / 215 /
// 218. Of E2M1, 256 rows pay where the second half is more than an eighth full, 160 and 512 rows each: 264 and 622 us,
// 363 and 760 with 128 (2048 -> 7168, 144 and 512: 163 and 373, 210 and 451); at 128 each they do by a tenth where no
// pair is masked (256 and 296 us) and lose where a quarter is (596 and 512). E4M3's fragments do not fit the registers at
// that height.
int tile_rows(int each, int element)
{
    if (each <= 48) return 64;
    return element == MOE_MX_E2M1 && each > 144 ? 256 : 128;
}

int check_mx(long long rows, int cols, int dtype, int element)
{
    if (rows < 0 || cols < kPiece || cols % kPiece) return MOE_ERR_SHAPE;
    if (dtype != MOE_FP16 && dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_DTYPE;
    if (element != MOE_MX_E2M1 && element != MOE_MX_E4M3) return MOE_ERR_QUANT;
    if (rows > kMaxBlocks / ((cols + kBlock - 1) / kBlock)) return MOE_ERR_SHAPE;
    return MOE_OK;
}

template <class F>
void by_type(int dtype, F f)
{
    if (dtype == MOE_FP16) f(F16());
    else if (dtype == MOE_BF16) f(BF16());
    else f(F32());
}

}  // namespace

extern "C" {

int moe_mx_quantize(const void *x, int64_t rows, int cols, int dtype, int element, void *codes, uint8_t *scales,
                    void *stream)
{
    const int rc = check_mx(rows, cols, dtype, element);
    if (rc) return rc;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_NULLPTR;
    if (!aligned(x, 16) || !aligned(codes, 16)) return MOE_ERR_ALIGN;
    MxArgs a;
    a.in = x;
    a.out = codes;
    a.scales_in = nullptr;
    a.scales_out = scales;
    a.per_row = cols / kPiece;
    a.blocks = (cols + kBlock - 1) / kBlock;
    a.pieces = rows * a.per_row;
    // An input that fills the Infinity Cache passes it by, which leaves the cache to the codes: bf16 [32768, 7168]
    // to E2M1 and back 202 us, 220 otherwise; [65536, 2048] to E4M3 64 us and 70. A smaller one may lie in it, fresh
    // from the kernel before: [32768, 2048] to E2M1 30 us past the cache, 28 through it.
    const bool once = rows * cols * (dtype == MOE_FP32 ? 4 : 2) >= kOnceBytes;
    const bool ragged = cols % kBlock != 0;
    const dim3 g((unsigned)((2 * rows * a.blocks + kMxThreads - 1) / kMxThreads)), b(kMxThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) {
        using T = decltype(type);
        auto launch = [&](auto e, auto half) {
            constexpr int kE = decltype(e)::value;
            constexpr bool kRagged = decltype(half)::value;
            if (once) hipLaunchKernelGGL((quantize_kernel<T, kE, kRagged, true>), g, b, 0, st, a);
            else hipLaunchKernelGGL((quantize_kernel<T, kE, kRagged, false>), g, b, 0, st, a);
        };
        using std::integral_constant;
        using Four = integral_constant<int, MOE_MX_E2M1>;
        using Eight = integral_constant<int, MOE_MX_E4M3>;
        if (element == MOE_MX_E2M1 && ragged) launch(Four(), std::true_type());
        else if (element == MOE_MX_E2M1) launch(Four(), std::false_type());
        else if (ragged) launch(Eight(), std::true_type());
        else launch(Eight(), std::false_type());
    });
    return launched();
}

int moe_mx_dequantize(const void *codes, const uint8_t *scales, int64_t rows, int cols, int dtype, int element,
                      void *out, void *stream)
{
    const int rc = check_mx(rows, cols, dtype, element);
    if (rc) return rc;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !out) return MOE_ERR_NULLPTR;
    if (!aligned(codes, 16) || !aligned(out, 16)) return MOE_ERR_ALIGN;
    MxArgs a;
    a.in = codes;
    a.out = out;
    a.scales_in = scales;
    a.scales_out = nullptr;
    a.per_row = cols / kPiece;
    a.blocks = (cols + kBlock - 1) / kBlock;
    a.pieces = rows * a.per_row;
    const bool ragged = cols % kBlock != 0;
    const dim3 g((unsigned)((a.pieces + kMxThreads - 1) / kMxThreads)), b(kMxThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) {
        using T = decltype(type);
        if (element == MOE_MX_E2M1 && ragged) hipLaunchKernelGGL((dequantize_kernel<T, MOE_MX_E2M1, true>), g, b, 0, st, a);
        else if (element == MOE_MX_E2M1) hipLaunchKernelGGL((dequantize_kernel<T, MOE_MX_E2M1, false>), g, b, 0, st, a);
        else if (ragged) hipLaunchKernelGGL((dequantize_kernel<T, MOE_MX_E4M3, true>), g, b, 0, st, a);
        else hipLaunchKernelGGL((dequantize_kernel<T, MOE_MX_E4M3, false>), g, b, 0, st, a);
    });
    return launched();
}

int moe_expert_product(const void *x, const uint8_t *x_scales, int element, const uint8_t *weights,
                       const uint8_t *weight_scales, const int32_t *ep_recv_count, int ep_world,
                       int experts_per_rank, int rows, int k, int n, int activation, int dtype, void *out,
                       void *stream)
{
    if (ep_world < kMinWorld || ep_world > kMaxWorld || experts_per_rank < 1 ||
        (long long)ep_world * experts_per_rank > kMaxExperts || rows < 0 || k < kPiece || k % kPiece || n < 1)
        return MOE_ERR_SHAPE;
    if (element != MOE_MX_E2M1 && element != MOE_MX_E4M3) return MOE_ERR_QUANT;
    if (dtype != MOE_FP16 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
    if (activation != MOE_ACT_NONE && activation != MOE_ACT_SWIGLU) return MOE_ERR_SHAPE;
    const bool glu = activation == MOE_ACT_SWIGLU;
    if (glu && n % 2) return MOE_ERR_SHAPE;
    ProductArgs a;
    a.W = ep_world;
    a.epr = experts_per_rank;
    a.E = ep_world * experts_per_rank;
    a.S = a.E;                                  // segments of a rank: experts_per_rank * ep_world
    a.rows = rows;
    a.k = k;
    a.n = n;
    a.nb = (k + kBlock - 1) / kBlock;
    a.fo = glu ? n / 2 : n;
    // offsets inside one expert's weights, and inside the rows of one tile, are 32-bit
    if ((long long)n * k > 4ll << 30 || k > 1 << 24) return MOE_ERR_SHAPE;
    const int each = rows / a.E;                // rows of an expert, were they even
    // rows and columns of a tile
    const int tall = tile_rows(each, element);
    const int cols = (tall == 64 ? 128 : 256) / (glu ? 2 : 1);
    a.ntiles = (a.fo + cols - 1) / cols;
    // a tile starts at every expert's first row, so at most this many
    const long long mtiles = rows / tall + std::min(a.E, rows);
    // rows and tiles are counted past the last one by up to a tile's height and a stride of the grid
    if (rows > INT_MAX - 256 || mtiles * a.ntiles > INT_MAX - kWorkgroupsSmall) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !x_scales || !weights || !weight_scales || !ep_recv_count || !out) return MOE_ERR_NULLPTR;
    if (!aligned(x, 16) || !aligned(weights, 16) || !aligned(ep_recv_count, 4) || !aligned(out, 2))
        return MOE_ERR_ALIGN;
    a.x = static_cast<const uint8_t *>(x);
    a.xs = x_scales;
    a.w = weights;
    a.ws = weight_scales;
    a.erc = ep_recv_count;
    a.out = out;
    const dim3 g((unsigned)std::min<long long>(mtiles * a.ntiles, tall == 64 ? kWorkgroupsSmall : kWorkgroupsLarge));
    const dim3 b(tall == 64 ? 256 : 512);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
#define MOE_PRODUCT_G(T, XF, G)                                                                       \
    do {                                                                                              \
        if (tall == 64) hipLaunchKernelGGL((expert_product_kernel<T, XF, 4, 2, 1, 4, 1, 4, G>), g, b, 0, st, a); \
        else if (XF == 4 && tall == 256)                                                              \
            hipLaunchKernelGGL((expert_product_kernel<T, 4, 8, 4, 2, 4, 2, 2, G>), g, b, 0, st, a);   \
        else hipLaunchKernelGGL((expert_product_kernel<T, XF, 4, 4, 2, 4, 2, 2, G>), g, b, 0, st, a); \
    } while (0)
#define MOE_PRODUCT(T, XF)                                                                            \
    do {                                                                                              \
        if (glu) MOE_PRODUCT_G(T, XF, true);                                                          \
        else MOE_PRODUCT_G(T, XF, false);                                                             \
    } while (0)
    if (dtype == MOE_FP16) {
        if (element == MOE_MX_E2M1) MOE_PRODUCT(F16, 4);
        else MOE_PRODUCT(F16, 0);
    } else {
        if (element == MOE_MX_E2M1) MOE_PRODUCT(BF16, 4);
        else MOE_PRODUCT(BF16, 0);
    }
#undef MOE_PRODUCT
#undef MOE_PRODUCT_G
    return launched();
}

}  // extern "C"
