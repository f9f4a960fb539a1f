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

namespace {

using namespace moe_detail;

constexpr int kBlock = 32;                 // elements that share a scale byte
constexpr int kPiece = 16;                 // elements a lane quantises: half a block
constexpr int kMxThreads = 256;
constexpr long long kMaxRows = (1ll << 31) - 1;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));      // loads and stores whose address has any alignment
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
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

// 16 elements of T from `p` (16-byte aligned: a row is a multiple of 16 elements)
template <class T>
__device__ __forceinline__ void load_piece(const void *in, long long piece, float (&x)[kPiece])
{
    const u32x4 *p = reinterpret_cast<const u32x4 *>(static_cast<const typename T::raw *>(in) + piece * kPiece);
    if constexpr (sizeof(typename T::raw) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const u32x4 v = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = __uint_as_float(v[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const u32x4 v = p[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[8 * i + 2 * j] = T::load((uint16_t)(v[j] & 0xffff));
                x[8 * i + 2 * j + 1] = T::load((uint16_t)(v[j] >> 16));
            }
        }
    }
}

// A lane takes 16 elements and its neighbour the block's other half; a row with a last block of 16 leaves that
// block to one lane. E: MOE_MX_E2M1 or MOE_MX_E4M3.
template <class T, int E, bool RAGGED>
__global__ __launch_bounds__(kMxThreads) void quantize_kernel(MxArgs a)
{
    const long long lane_piece = (long long)blockIdx.x * kMxThreads + threadIdx.x;
    // RAGGED: the grid counts two pieces for every block, and the half that a row's last block lacks is empty
    long long row = 0, piece = lane_piece;
    bool live;
    if (RAGGED) {
        row = lane_piece / (2 * a.blocks);
        const int q = (int)(lane_piece - row * (2 * a.blocks));
        piece = row * a.per_row + q;
        live = piece < a.pieces && q < a.per_row;
    } else {
        live = piece < a.pieces;
    }
    float x[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = 0.f;
    if (live) load_piece<T>(a.in, piece, x);
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
    const long long piece = (long long)blockIdx.x * kMxThreads + threadIdx.x;
    if (piece >= a.pieces) return;
    long long block = piece / 2;
    if (RAGGED) {
        const long long row = piece / a.per_row;
        block = row * a.blocks + (piece - row * a.per_row) / 2;
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

constexpr int kProductThreads = 256;       // four wavefronts
constexpr int kMaxExperts = 1024;          // dispatch's limits
constexpr int kMinWorld = 2, kMaxWorld = 768;
constexpr int kStep = 128;                 // elements of k in one matrix instruction
constexpr int kSuper = 4 * kStep;          // ... in a group of four, whose 16 scale bytes are one load
constexpr int kWorkgroups = 1024;          // at most: every CU's fill, with tiles to spare for none
constexpr int kFrags = 4;                  // 16-wide weight fragments of a workgroup

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
    uint32_t part[2][kProductThreads / kWave];
    int expert;
};

// Fills the plan for tiles of BM rows and returns their number. The counts are ep_recv_count's differences, held
// within [0, rows] whatever the array holds. All threads call it.
template <int BM>
__device__ int make_plan(const ProductArgs &a, Plan &plan)
{
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    constexpr int kEach = kMaxExperts / kProductThreads;
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
    // rows before this thread's experts (sums that stop at `rows`, which keeps them in 32 bits and in order)
    uint32_t inc = sum;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t v = __shfl_up(inc, d);
        if (lane >= d) inc = min(most, inc + v);
    }
    if (lane == kWave - 1) plan.part[0][wave] = inc;
    uint32_t before = __shfl_up(inc, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    for (int i = 0; i < wave; ++i) before = min(most, before + plan.part[0][i]);
    uint32_t start[kEach + 1], tiles = 0;
    start[0] = before;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        start[i + 1] = min(most, start[i] + count[i]);
        tiles += (start[i + 1] - start[i] + BM - 1) / BM;
    }
    inc = tiles;
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) {
        const uint32_t v = __shfl_up(inc, d);
        if (lane >= d) inc += v;
    }
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
    if (tid == kProductThreads - 1) {
        plan.row[kMaxExperts] = start[kEach];
        plan.tile[kMaxExperts] = at;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(plan.tile[kMaxExperts]);
}

// Row tile `mt` of the plan (below its number of tiles). All threads call it; it holds a barrier.
template <int BM>
__device__ Tile find_tile(Plan &plan, int mt)
{
    const int tid = threadIdx.x;
    for (int e = tid; e < kMaxExperts; e += kProductThreads)
        if (plan.tile[e] <= (uint32_t)mt && (uint32_t)mt < plan.tile[e + 1]) plan.expert = e;
    __syncthreads();
    const int e = __builtin_amdgcn_readfirstlane(plan.expert);
    return Tile{e, (int)__builtin_amdgcn_readfirstlane(plan.row[e] + (mt - plan.tile[e]) * BM),
                (int)__builtin_amdgcn_readfirstlane(plan.row[e + 1])};
}

// One 16 x 16 x 128 step: weights (E2M1) by rows of elements of format XF (0: E4M3, 4: E2M1), the scale bytes in
// byte SEL of ws and xs. Lane (r, g), r = lane % 16, g = lane / 16, holds 32 elements of row r and the scale of
// its row's block g: E2M1 elements 32g..32g+31; E4M3 elements 16g..16g+15 and 64+16g..64+16g+15. Result register
// i is weight row 4g + i, input row r.
template <int XF, int SEL>
__device__ __forceinline__ f32x4 mma(i32x8 w, i32x8 x, f32x4 c, uint32_t ws, uint32_t xs)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 4, XF, SEL, (int)ws, SEL, (int)xs);
}

__device__ __forceinline__ i32x8 join(u32x4 lo, u32x4 hi)
{
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// The 32 elements of a step that starts at element `at` of a row, whole
template <int XF>
__device__ __forceinline__ i32x8 load_step(const uint8_t *row, int at, int g)
{
    if constexpr (XF == 4) {
        const u32x4 v = *reinterpret_cast<const u32x4_a8 *>(row + (at + 32 * g) / 2);
        return join(v, v);
    } else {
        return join(*reinterpret_cast<const u32x4 *>(row + at + 16 * g),
                    *reinterpret_cast<const u32x4 *>(row + at + 64 + 16 * g));
    }
}
// ... with zeros past the row's k elements
template <int XF>
__device__ __forceinline__ i32x8 load_last(const uint8_t *row, int at, int g, int k)
{
    u32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    if constexpr (XF == 4) {
        const int p = at + 32 * g;
        if (p + 32 <= k) lo = *reinterpret_cast<const u32x4_a8 *>(row + p / 2);
        else if (p < k) {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(row + p / 2);
            lo[0] = v[0];
            lo[1] = v[1];
        }
    } else {
        if (at + 16 * g < k) lo = *reinterpret_cast<const u32x4 *>(row + at + 16 * g);
        if (at + 64 + 16 * g < k) hi = *reinterpret_cast<const u32x4 *>(row + at + 64 + 16 * g);
    }
    return join(lo, hi);
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
// The scale bytes of a lane's blocks in four steps: byte g of each word of the row's 16 bytes, one word
__device__ __forceinline__ uint32_t load_scales(const uint8_t *p, uint32_t sel)
{
    const u32x4 d = *reinterpret_cast<const u32x4_a1 *>(p);
    return __builtin_amdgcn_perm(d[1], d[0], sel) | (__builtin_amdgcn_perm(d[3], d[2], sel) << 16);
}
// ... for every g: a transpose of 4 x 4 bytes
__device__ __forceinline__ u32x4 by_group(u32x4 d)
{
    const uint32_t a = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), b = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u), e = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
    return u32x4{__builtin_amdgcn_perm(b, a, 0x05040100u), __builtin_amdgcn_perm(b, a, 0x07060302u),
                 __builtin_amdgcn_perm(e, c, 0x05040100u), __builtin_amdgcn_perm(e, c, 0x07060302u)};
}

template <class T>
__device__ __forceinline__ void store_out(const ProductArgs &a, int row, int col, f32x4 v)
{
    typename T::raw *p = static_cast<typename T::raw *>(a.out) + (size_t)row * a.fo + col;
    if (col + 4 <= a.fo && a.fo % 4 == 0) {
        u32x2 u;
        u[0] = (uint32_t)T::store(v[0]) | ((uint32_t)T::store(v[1]) << 16);
        u[1] = (uint32_t)T::store(v[2]) | ((uint32_t)T::store(v[3]) << 16);
        *reinterpret_cast<u32x2_a1 *>(p) = u;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < a.fo) p[i] = T::store(v[i]);
    }
}

// silu(gate) * up by the hardware's exponential and reciprocal (an ulp each; the exponent's argument is off by |gate|
// half steps): far below the 16-bit rounding behind it
__device__ __forceinline__ float swiglu(float gate, float up)
{
    return gate * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(gate * -1.44269504f)) * up;
}

// Rows of one expert, 16 * FR at a time, against 64 weight rows (32 of the gate's and 32 of the up projection's
// with GLU). The four wavefronts share out k in supersteps of 512 and add up in LDS, wavefront 0's part first.
template <class T, int XF, int FR, bool GLU>
__global__ __launch_bounds__(kProductThreads) void expert_product_kernel(ProductArgs a)
{
    __shared__ Plan plan;
    __shared__ f32x4 part[kProductThreads / kWave][kFrags][kWave];
    const int total = make_plan<FR * 16>(a, plan) * a.ntiles;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int nt = t % a.ntiles;
    const Tile tile = find_tile<FR * 16>(plan, t / a.ntiles);
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int r = lane % 16, g = lane / 16;
    constexpr int kOut = GLU ? kFrags / 2 : kFrags;          // output fragments of 16 columns
    const int half = a.n / 2, col0 = nt * kOut * 16;
    const size_t wrow = (size_t)a.k / 2, xrow = XF == 4 ? (size_t)a.k / 2 : (size_t)a.k;
    const uint8_t *wp[kFrags], *wsp[kFrags], *xp[FR], *xsp[FR];
#pragma unroll
    for (int j = 0; j < kFrags; ++j) {
        // columns past the last one read the last one's weights; their results are not stored
        const int c = min(col0 + (j % kOut) * 16 + r, a.fo - 1);
        const size_t row = (size_t)tile.expert * a.n + (GLU && j >= kOut ? half : 0) + c;
        wp[j] = a.w + row * wrow;
        wsp[j] = a.ws + row * a.nb;
    }
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const size_t row = min(tile.row + f * 16 + r, tile.end - 1);
        xp[f] = a.x + row * xrow;
        xsp[f] = a.xs + row * a.nb;
    }
    f32x4 acc[FR][kFrags];
#pragma unroll
    for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int j = 0; j < kFrags; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const uint32_t sel = 0x0c0c0400u + 0x0101u * g;           // byte g of the low word, byte g of the high word
    const int supers = a.k / kSuper;
    for (int s = wave; s < supers; s += kProductThreads / kWave) {
        uint32_t ws[kFrags], xs[FR];
#pragma unroll
        for (int j = 0; j < kFrags; ++j) ws[j] = load_scales(wsp[j] + 16 * s, sel);
#pragma unroll
        for (int f = 0; f < FR; ++f) xs[f] = load_scales(xsp[f] + 16 * s, sel);
#define MOE_STEP(I)                                                                                   \
        {                                                                                             \
            i32x8 wf[kFrags], xf[FR];                                                                 \
            _Pragma("unroll") for (int j = 0; j < kFrags; ++j)                                        \
                wf[j] = load_step<4>(wp[j], kSuper * s + kStep * I, g);                               \
            _Pragma("unroll") for (int f = 0; f < FR; ++f)                                            \
                xf[f] = load_step<XF>(xp[f], kSuper * s + kStep * I, g);                              \
            _Pragma("unroll") for (int f = 0; f < FR; ++f)                                            \
                _Pragma("unroll") for (int j = 0; j < kFrags; ++j)                                    \
                    acc[f][j] = mma<XF, I>(wf[j], xf[f], acc[f][j], ws[j], xs[f]);                    \
        }
        MOE_STEP(0)
        MOE_STEP(1)
        MOE_STEP(2)
        MOE_STEP(3)
#undef MOE_STEP
    }
    // the last k % 512 elements, one step to a wavefront in turn
    for (int at = supers * kSuper + kStep * wave; at < a.k; at += kSuper) {
        const int b = at / kBlock + g;
        i32x8 wf[kFrags], xf[FR];
        uint32_t ws[kFrags], xs[FR];
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
            wf[j] = load_last<4>(wp[j], at, g, a.k);
            ws[j] = b < a.nb ? wsp[j][b] : 127;
        }
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            xf[f] = load_last<XF>(xp[f], at, g, a.k);
            xs[f] = b < a.nb ? xsp[f][b] : 127;
        }
#pragma unroll
        for (int f = 0; f < FR; ++f)
#pragma unroll
            for (int j = 0; j < kFrags; ++j) acc[f][j] = mma<XF, 0>(wf[j], xf[f], acc[f][j], ws[j], xs[f]);
    }

#pragma unroll
    for (int f = 0; f < FR; ++f) {
        if (f) __syncthreads();
#pragma unroll
        for (int j = 0; j < kFrags; ++j) part[wave][j][lane] = acc[f][j];
        __syncthreads();
        if (wave < kOut) {
            f32x4 v = part[0][wave][lane];
#pragma unroll
            for (int i = 1; i < kProductThreads / kWave; ++i) v += part[i][wave][lane];
            if (GLU) {
                f32x4 u = part[0][wave + kOut][lane];
#pragma unroll
                for (int i = 1; i < kProductThreads / kWave; ++i) u += part[i][wave + kOut][lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], u[i]);
            }
            const int row = tile.row + f * 16 + r, col = col0 + wave * 16 + 4 * g;
            if (row < tile.end && col < a.fo) store_out<T>(a, row, col, v);
        }
    }
    __syncthreads();
    }
}

// Rows of one expert, 16 * FR * WM at a time, against 16 * NF * WN weight rows (half of them the gate's, half the
// matching ones of the up projection with GLU): WM x WN wavefronts, each with FR x NF fragments of its own and all of k.
//
// Both sides go through LDS: a matrix instruction's lane holds 16 bytes of a row whose neighbours sit in lanes 16
// apart, so loading straight into its layout makes the cache look at every lane's 16 bytes by itself (one look-up a
// clock), where eight adjacent lanes that read a line of 128 bytes count as one. A stage is 128 bytes of an input
// row, kSub instruction steps: 256 elements of E2M1, 128 of E4M3. The 16-byte pieces of a row are swapped by its number
// so that the eight lanes that LDS serves in a clock meet every bank once, writing and reading.
//
// A stage's pieces are fetched into registers two stages ahead and written to the idle half of LDS one ahead, a few
// between each fragment's matrix instructions, so that those never run dry. Input fragments are read two ahead. The
// barrier comes when the current half has been read, two fragments before a stage's end; the next stage's first
// fragments are read behind it while those two multiply. Scale bytes come 512 elements (four steps) at a time and
// become a word per (row, g) on the way.
template <class T, int XF, int FR, int NF, int WM, bool GLU>
__global__ __launch_bounds__(kProductThreads, FR *NF <= 16 ? 2 : 1) void expert_product_wide_kernel(ProductArgs a)
{
    constexpr int kWaves = kProductThreads / kWave, WN = kWaves / WM, kRowsW = WN * NF * 16, kRowsX = WM * FR * 16;
    constexpr int kSub = XF == 4 ? 2 : 1, kStages = 4 / kSub;  // steps of a stage, stages of 512 elements
    constexpr int kPw = 4 * kSub, kPx = 8;                    // 16-byte pieces of a row in a stage
    constexpr int kLoadsW = kRowsW * kPw / kProductThreads, kLoadsX = kRowsX * kPx / kProductThreads;
    constexpr int kLoads = kLoadsW + kLoadsX;
    constexpr int kScalesW = kRowsW / kProductThreads;        // scale rows of the weights that a thread carries
    static_assert(kRowsW % kProductThreads == 0 && kRowsX <= kProductThreads, "whole scale rows a thread");
    static_assert(kRowsX * kPx % kProductThreads == 0, "every thread carries as many pieces");
    __shared__ Plan plan;
    __shared__ u32x4 wl[2][kRowsW * kPw], xl[2][kRowsX * kPx], wsl[2][kRowsW], xsl[2][kRowsX];

    const int total = make_plan<kRowsX>(a, plan) * a.ntiles;
    for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int nt = t % a.ntiles;
    const Tile tile = find_tile<kRowsX>(plan, t / a.ntiles);
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), wm = wave / WN, wn = wave % WN;
    const int r = lane % 16, g = lane / 16;
    constexpr int kOut = GLU ? NF / 2 : NF, kOwn = NF * 16;   // output fragments and weight rows of a wavefront
    const int half = a.n / 2, tile0 = nt * WN * kOut * 16;
    const uint32_t wrow = a.k / 2, xrow = XF == 4 ? a.k / 2 : a.k;
    const uint8_t *wb = a.w + (size_t)tile.expert * a.n * wrow, *wsb = a.ws + (size_t)tile.expert * a.n * a.nb;
    const uint8_t *xb = a.x + (size_t)tile.row * xrow, *xsb = a.xs + (size_t)tile.row * a.nb;
    const int last = tile.end - 1 - tile.row;                 // rows past the expert's last read the last one
    // weight row of a place in the tile; columns past the last one read the last one's, and are not stored
    auto weight_row = [&](int q) -> uint32_t {
        const int c = GLU ? q / kOwn * (kOwn / 2) + q % (kOwn / 2) : q;
        return (GLU && q % kOwn >= kOwn / 2 ? half : 0) + min(tile0 + c, a.fo - 1);
    };
    // piece p of row q in LDS, for rows of 4 and of 8 pieces
    auto place4 = [](int q, int p) { return q * 4 + (p ^ ((q >> 1) & 3)); };
    auto place8 = [](int q, int p) { return q * 8 + (p ^ (q & 7)); };
    // this thread's pieces: where in a row's stage, and the place in LDS (piece i: kProductThreads * i further)
    uint32_t wo[kLoadsW], xo[kLoadsX];
#pragma unroll
    for (int i = 0; i < kLoadsW; ++i) wo[i] = weight_row((tid + i * kProductThreads) / kPw) * wrow + 16 * (tid % kPw);
#pragma unroll
    for (int i = 0; i < kLoadsX; ++i) xo[i] = (uint32_t)min((tid + i * kProductThreads) / kPx, last) * xrow + 16 * (tid % kPx);
    const int wat = kSub == 2 ? place8(tid / 8, tid % 8) : place4(tid / 4, tid % 4), xat = place8(tid / 8, tid % 8);
    uint32_t wso[kScalesW];
#pragma unroll
    for (int i = 0; i < kScalesW; ++i) wso[i] = weight_row(tid + i * kProductThreads) * a.nb;
    const uint32_t xso = (uint32_t)min(tid % kRowsX, last) * a.nb;
    // a reader's pieces: of fragment 0, the others lie 16 rows apart
    const int lo = place8(r, g), hi = place8(r, 4 + g);
    const int wfrag[2] = {wn * kOwn * kPw + (kSub == 2 ? lo : place4(r, g)), wn * kOwn * kPw + hi};
    const int xfrag[2] = {wm * FR * 16 * kPx + lo, wm * FR * 16 * kPx + hi};

    f32x4 acc[FR][NF];
#pragma unroll
    for (int f = 0; f < FR; ++f)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int supers = a.k / kSuper, stages = supers * kStages;
    u32x4 piece[kLoads], wsr[kScalesW], xsr;
    // Loads of whole stages. Beyond the last one the last one is read again, and not used: a branch here would make
    // the compiler wait for the load at its end.
    auto load = [&](int i, int stage) {
        const uint32_t at = min(stage, stages - 1);
        if (i < kLoadsW) piece[i] = *reinterpret_cast<const u32x4_a8 *>(wb + (wo[i] + at * (16 * kPw)));
        else piece[i] = *reinterpret_cast<const u32x4_a8 *>(xb + (xo[i - kLoadsW] + at * (16 * kPx)));
    };
    auto keep = [&](int i, int buf) {
        if (i < kLoadsW) wl[buf][wat + i * kProductThreads] = piece[i];
        else xl[buf][xat + (i - kLoadsW) * kProductThreads] = piece[i];
    };
    auto load_scales = [&](int super) {
        const uint32_t at = min(super, supers - 1) * 16;
#pragma unroll
        for (int i = 0; i < kScalesW; ++i) wsr[i] = *reinterpret_cast<const u32x4_a1 *>(wsb + (wso[i] + at));
        xsr = *reinterpret_cast<const u32x4_a1 *>(xsb + (xso + at));
    };
    auto keep_scales = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kScalesW; ++i) wsl[buf][tid + i * kProductThreads] = by_group(wsr[i]);
        xsl[buf][tid % kRowsX] = by_group(xsr);          // threads of the same row write the same bytes
    };
    const uint32_t *wsw = reinterpret_cast<const uint32_t *>(wsl) + (wn * kOwn + r) * 4 + g;
    const uint32_t *xsw = reinterpret_cast<const uint32_t *>(xsl) + (wm * FR * 16 + r) * 4 + g;
    i32x8 wf[2][NF], xf[FR];
    uint32_t ws[NF], xs[FR];
    // fragments of step i of 512 elements
    auto read_w = [&](int i) {
        const u32x4 *l = wl[i / kSub & 1] + wfrag[i % kSub];
#pragma unroll
        for (int j = 0; j < NF; ++j) wf[i & 1][j] = join(l[j * 16 * kPw], l[j * 16 * kPw]);
    };
    auto read_x = [&](int i, int f) {
        const u32x4 *l = xl[i / kSub & 1] + f * 16 * kPx;
        xf[f] = XF == 4 ? join(l[xfrag[i % kSub]], l[xfrag[i % kSub]]) : join(l[xfrag[0]], l[xfrag[1]]);
    };
    auto read_scales = [&](int buf) {
#pragma unroll
        for (int j = 0; j < NF; ++j) ws[j] = wsw[buf * kRowsW * 4 + j * 64];
#pragma unroll
        for (int f = 0; f < FR; ++f) xs[f] = xsw[buf * kRowsX * 4 + f * 64];
    };
    if (supers > 0) {
        load_scales(0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load(i, 0);
        keep_scales(0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) keep(i, 0);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) load(i, 1);
        __syncthreads();
        read_w(0);
        read_x(0, 0);
        read_x(0, 1);
        read_scales(0);
    }
    for (int super = 0; super < supers; ++super) {
#define MOE_WIDE_STEP(I)                                                                              \
        {                                                                                             \
            constexpr int kStage = I / kSub, kGroups = (FR - 2) * kSub;                               \
            if (I == 1) load_scales(super + 1);                                                       \
            if (I == 3) keep_scales((super + 1) & 1);                                                 \
            _Pragma("unroll") for (int f = 0; f < FR - 2; ++f) {                                      \
                const int group = I % kSub * (FR - 2) + f;                                            \
                read_x(I, f + 2);                                                                     \
                _Pragma("unroll") for (int i = group * kLoads / kGroups; i < (group + 1) * kLoads / kGroups; ++i) { \
                    keep(i, (kStage + 1) & 1);                                                        \
                    load(i, super * kStages + kStage + 2);                                            \
                }                                                                                     \
                _Pragma("unroll") for (int j = 0; j < NF; ++j)                                        \
                    acc[f][j] = mma<XF, I>(wf[I & 1][j], xf[f], acc[f][j], ws[j], xs[f]);             \
                __builtin_amdgcn_sched_barrier(0);                                                    \
            }                                                                                         \
            if (I % kSub == kSub - 1) __syncthreads();                                                \
            __builtin_amdgcn_sched_barrier(0);                                                        \
            read_w((I + 1) & 3);                                                                      \
            read_x((I + 1) & 3, 0);                                                                   \
            read_x((I + 1) & 3, 1);                                                                   \
            __builtin_amdgcn_sched_barrier(0);                                                        \
            _Pragma("unroll") for (int f = FR - 2; f < FR; ++f)                                       \
                _Pragma("unroll") for (int j = 0; j < NF; ++j)                                        \
                    acc[f][j] = mma<XF, I>(wf[I & 1][j], xf[f], acc[f][j], ws[j], xs[f]);             \
            if (I == 3) read_scales((super + 1) & 1);                                                 \
            __builtin_amdgcn_sched_barrier(0);                                                        \
        }
        MOE_WIDE_STEP(0)
        MOE_WIDE_STEP(1)
        MOE_WIDE_STEP(2)
        MOE_WIDE_STEP(3)
#undef MOE_WIDE_STEP
    }
    // the last k % 512 elements, a step at a time
    for (int at = supers * kSuper; at < a.k; at += kStep) {
        __syncthreads();
        constexpr int kTx = XF == 4 ? 4 : 8;                  // pieces of an input row in one step
#pragma unroll 1
        for (int c = tid; c < kRowsW * 4; c += kProductThreads)
            wl[0][kSub == 2 ? place8(c / 4, c % 4) : place4(c / 4, c % 4)] =
                load_piece_or_zero<4>(wb + weight_row(c / 4) * wrow + 16 * (c % 4), at, c % 4, a.k);
#pragma unroll 1
        for (int c = tid; c < kRowsX * kTx; c += kProductThreads)
            xl[0][place8(c / kTx, c % kTx)] =
                load_piece_or_zero<XF>(xb + (uint32_t)min(c / kTx, last) * xrow + 16 * (c % kTx), at, c % kTx, a.k);
        const int b = at / kBlock;
        u32x4 v;
#pragma unroll
        for (int j = 0; j < kScalesW; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = b + i < a.nb ? wsb[wso[j] + b + i] : 127;
            wsl[0][tid + j * kProductThreads] = v;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = b + i < a.nb ? xsb[xso + b + i] : 127;
        xsl[0][tid % kRowsX] = v;
        __syncthreads();
        read_w(0);
        read_scales(0);
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            read_x(0, f);
#pragma unroll
            for (int j = 0; j < NF; ++j) acc[f][j] = mma<XF, 0>(wf[0][j], xf[f], acc[f][j], ws[j], xs[f]);
        }
    }
#pragma unroll
    for (int f = 0; f < FR; ++f) {
        const int row = tile.row + (wm * FR + f) * 16 + r;
        if (row >= tile.end) continue;
#pragma unroll
        for (int j = 0; j < kOut; ++j) {
            f32x4 v = acc[f][j];
            if (GLU) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = swiglu(v[i], acc[f][j + kOut][i]);
            }
            const int col = tile0 + (wn * kOut + j) * 16 + 4 * g;
            if (col < a.fo) store_out<T>(a, row, col, v);
        }
    }
    __syncthreads();
    }
}

int check_mx(long long rows, int cols, int dtype, int element)
{
    if (rows < 0 || rows > kMaxRows || cols < kPiece || cols % kPiece) return MOE_ERR_SHAPE;
    if (dtype != MOE_FP16 && dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_DTYPE;
    if (element != MOE_MX_E2M1 && element != MOE_MX_E4M3) return MOE_ERR_QUANT;
    // two pieces a block, one piece a thread
    if (rows * ((cols + kBlock - 1) / kBlock) > (long long)INT_MAX * (kMxThreads / 2)) return MOE_ERR_SHAPE;
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
    const bool ragged = cols % kBlock != 0;
    const dim3 g((unsigned)((2 * rows * a.blocks + kMxThreads - 1) / kMxThreads)), b(kMxThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) {
        using T = decltype(type);
        if (element == MOE_MX_E2M1 && ragged) hipLaunchKernelGGL((quantize_kernel<T, MOE_MX_E2M1, true>), g, b, 0, st, a);
        else if (element == MOE_MX_E2M1) hipLaunchKernelGGL((quantize_kernel<T, MOE_MX_E2M1, false>), g, b, 0, st, a);
        else if (ragged) hipLaunchKernelGGL((quantize_kernel<T, MOE_MX_E4M3, true>), g, b, 0, st, a);
        else hipLaunchKernelGGL((quantize_kernel<T, MOE_MX_E4M3, false>), g, b, 0, st, a);
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
    const int tall = each <= 8 ? 16 : (each <= 40 ? 64 : (each <= 150 ? 128 : 192));
    const int cols = (tall == 16 ? kFrags * 16 : 256) / (glu ? 2 : 1);
    a.ntiles = (a.fo + cols - 1) / cols;
    // a tile starts at every expert's first row, so at most this many
    const long long mtiles = rows / tall + std::min(a.E, rows);
    if (mtiles * a.ntiles > INT_MAX) return MOE_ERR_SHAPE;
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
    const dim3 g((unsigned)std::min<long long>(mtiles * a.ntiles, kWorkgroups)), b(kProductThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
#define MOE_PRODUCT_G(T, XF, G)                                                                       \
    do {                                                                                              \
        if (tall == 16) hipLaunchKernelGGL((expert_product_kernel<T, XF, 1, G>), g, b, 0, st, a);     \
        else if (tall == 64) hipLaunchKernelGGL((expert_product_wide_kernel<T, XF, 4, 4, 1, G>), g, b, 0, st, a); \
        else if (tall == 128) hipLaunchKernelGGL((expert_product_wide_kernel<T, XF, 4, 8, 2, G>), g, b, 0, st, a); \
        else hipLaunchKernelGGL((expert_product_wide_kernel<T, XF, 6, 8, 2, G>), g, b, 0, st, a);     \
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
