// moe_int8.hip -- rows of 8-bit integers with a scale each, and the experts' product on them (gfx950, wave64).
//
//   quantise    scale = max|x| / 127 over the row, code = x / scale rounded to the nearest integer, ties to even
//   dequantise  code * scale
//   product     out[row] = act(xs[row] * ws[e, n] * sum_k x[row, k] * w[e, n, k]), e the expert that ep_recv_count gives
//               `row`; the sum is exact in 32-bit integers, the rest is fp32, rounded once.

#include "moe_rows.h"

#include <limits.h>

#include <algorithm>
#include <type_traits>

namespace {

using namespace moe_detail;

constexpr int kPiece = 16;                 // codes of 16 bytes
constexpr int kRowThreads = 256;
constexpr long long kOnceBytes = 256ll << 20;      // the Infinity Cache

typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

// --------------------------------------------------------------------------
// quantise and dequantise
// --------------------------------------------------------------------------

struct RowsArgs {
    const void *in;
    void *out;
    const float *scales_in;
    float *scales_out;
    long long rows;
    int cols, per_row;         // elements and pieces (the last one may be shorter) of a row
};

// Elements of a piece, `live` of them (0 to 16), zeros behind. Rows start at any element. ONCE: past the caches.
template <class T, bool ONCE>
__device__ __forceinline__ void load_piece(const typename T::raw *p, int live, float (&x)[kPiece])
{
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = 0.f;
    if (live == kPiece) {
        if constexpr (sizeof(typename T::raw) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u32x4_a4 *q = reinterpret_cast<const u32x4_a4 *>(p) + i;
                const u32x4 v = ONCE ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
                for (int j = 0; j < 4; ++j) x[4 * i + j] = T::load(v[j]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const u32x4_a2 *q = reinterpret_cast<const u32x4_a2 *>(p) + i;
                const u32x4 v = ONCE ? __builtin_nontemporal_load(q) : *q;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = T::load((uint16_t)(v[j] & 0xffff));
                    x[8 * i + 2 * j + 1] = T::load((uint16_t)(v[j] >> 16));
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (i < live) x[i] = T::load(p[i]);
    }
}
template <class T>
__device__ __forceinline__ void store_piece(typename T::raw *p, int live, const float (&x)[kPiece])
{
    if (live == kPiece) {
        if constexpr (sizeof(typename T::raw) == 4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = T::store(x[4 * i + j]);
                reinterpret_cast<u32x4_a4 *>(p)[i] = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u32x4 v;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = (uint32_t)T::store(x[8 * i + 2 * j]) | ((uint32_t)T::store(x[8 * i + 2 * j + 1]) << 16);
                reinterpret_cast<u32x4_a2 *>(p)[i] = v;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (i < live) p[i] = T::store(x[i]);
    }
}

// The codes of a piece, four a word. FAST, for 16-bit types and scale >= 2^-100: one correction step gives the
// correctly rounded quotient as far as its rounding to an integer goes, and adding 1.5 * 2^23 rounds it, ties to even,
// with the code in the low byte; both hold for every pair of 16-bit x and max|x| (checked exhaustively by the test of
// dispatch's quantiser, whose codes these are). Otherwise the division itself.
template <bool FAST>
__device__ __forceinline__ u32x4 codes_of(const float (&x)[kPiece], float scale, float inv)
{
    u32x4 c = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kPiece; ++i) {
        uint32_t q;
        if (FAST) {
            const float q0 = x[i] * inv, r = __builtin_fmaf(-q0, scale, x[i]);
            q = __float_as_uint(__builtin_fmaf(r, inv, q0) + 0x1.8p23f);
        } else {
            q = (uint32_t)(int)fminf(fmaxf(__builtin_rintf(x[i] / scale), -127.f), 127.f);
        }
        c[i / 4] |= (q & 0xffu) << (i % 4 * 8);
    }
    return c;
}

// The largest magnitude of a row over its lanes (16 or 64 of a wavefront, or the workgroup's four wavefronts).
template <int LANES>
__device__ __forceinline__ float row_max(float v, float (&part)[kRowThreads / kWave])
{
    if constexpr (LANES == 16) return wave_max<16>(v);
    v = wave_max(v);
    if constexpr (LANES == kRowThreads) {
        if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = v;
        __syncthreads();
        v = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
        __syncthreads();
    }
    return v;
}

// A row's LANES lanes hold it, J pieces each (J = 0: any number, read a second time for the codes, through the cache).
//
// Memory bounds it: 3 bytes an element of 16 bits, against some twelve instructions. bf16 [32768, 7168] 115 us, 6.1
// TB/s of 0.7 GB; [256, 2048] 3 us. Lanes by the row's pieces: 16 (four rows a wavefront), 64, or the workgroup's 256
// above 256 pieces: a wavefront that holds 448 pieces, 7 a lane, takes 173 us for 115. fp32 rows, which are divided in full,
// 285 us, 4.1 TB/s of 1.2 GB (weights, 256 x 4096 rows of 7168: 9.0 ms for 37.6 GB; [4096, 7168] 28 us).
template <class T, int LANES, int J, bool ONCE>
__global__ __launch_bounds__(kRowThreads) void quantize_kernel(RowsArgs a)
{
    constexpr int kRows = kRowThreads / LANES, kHeld = J ? J : 1;
    __shared__ float part[kRowThreads / kWave];
    const int lane = threadIdx.x % LANES;
    for (long long base = (long long)blockIdx.x * kRows; base < a.rows; base += (long long)gridDim.x * kRows) {
        const long long row = base + threadIdx.x / LANES;
        const bool live = row < a.rows;
        const typename T::raw *in = static_cast<const typename T::raw *>(a.in) + (live ? row : 0) * a.cols;
        float x[kHeld][kPiece];
        // magnitudes by their bits: ordered like the values, infinity and NaN above them all
        uint32_t top = 0;
        const int pieces = J ? J : (a.per_row + LANES - 1) / LANES;
#pragma unroll kHeld
        for (int j = 0; j < pieces; ++j) {
            const int p = lane + j * LANES;
            float(&v)[kPiece] = x[J ? j : 0];
            load_piece<T, ONCE>(in + (size_t)min(p, a.per_row) * kPiece,
                                live ? min(max(a.cols - p * kPiece, 0), kPiece) : 0, v);
#pragma unroll
            for (int i = 0; i < kPiece; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
        }
        // infinity stands for NaN too: fmax drops NaN
        const float most = row_max<LANES>(__uint_as_float(min(top, 0x7f800000u)), part);
        const bool finite = most < __builtin_huge_valf();
        const float scale = finite ? most / 127.f : __builtin_nanf("");
        const float inv = 1.f / scale;
        const bool some = finite && scale > 0.f, fast = sizeof(typename T::raw) == 2 && scale >= 0x1p-100f;
        if (live && lane == 0) a.scales_out[row] = scale;
#pragma unroll kHeld
        for (int j = 0; j < pieces; ++j) {
            const int p = lane + j * LANES, n = live ? min(max(a.cols - p * kPiece, 0), kPiece) : 0;
            float(&v)[kPiece] = x[J ? j : 0];
            if (!J) load_piece<T, ONCE>(in + (size_t)min(p, a.per_row) * kPiece, n, v);
            u32x4 c = {0, 0, 0, 0};
            if (some) c = fast ? codes_of<true>(v, scale, inv) : codes_of<false>(v, scale, inv);
            uint8_t *out = static_cast<uint8_t *>(a.out) + row * a.cols + (size_t)p * kPiece;
            if (n == kPiece) {
                *reinterpret_cast<u32x4_a1 *>(out) = c;
            } else {
#pragma unroll
                for (int i = 0; i < kPiece; ++i)
                    if (i < n) out[i] = (uint8_t)(c[i / 4] >> (i % 4 * 8));
            }
        }
    }
}

// A lane takes a piece. bf16 [32768, 7168] 125 to 140 us, 5.1 to 5.6 TB/s; stores past the caches 171.
template <class T>
__global__ __launch_bounds__(kRowThreads) void dequantize_kernel(RowsArgs a)
{
    const uint32_t q = blockIdx.x * kRowThreads + threadIdx.x, row = q / (uint32_t)a.per_row, p = q - row * a.per_row;
    if (row >= a.rows) return;
    const int live = min(a.cols - (int)p * kPiece, kPiece);
    const uint8_t *in = static_cast<const uint8_t *>(a.in) + (size_t)row * a.cols + (size_t)p * kPiece;
    u32x4 c = {0, 0, 0, 0};
    if (live == kPiece) {
        c = *reinterpret_cast<const u32x4_a1 *>(in);
    } else {
#pragma unroll
        for (int i = 0; i < kPiece; ++i)
            if (i < live) c[i / 4] |= (uint32_t)in[i] << (i % 4 * 8);
    }
    const float scale = a.scales_in[row];
    float x[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) x[i] = product((float)(int8_t)(c[i / 4] >> (i % 4 * 8)), scale);
    store_piece<T>(static_cast<typename T::raw *>(a.out) + (size_t)row * a.cols + (size_t)p * kPiece, live, x);
}

// --------------------------------------------------------------------------
// the experts' product
// --------------------------------------------------------------------------

struct ProductArgs {
    const uint8_t *x, *w;
    const float *xs, *ws;
    const int32_t *erc;
    void *out;
    int W, epr, E, S, rows, k, n, fo;      // fo: columns of out
    int ntiles;
};

// Rows of one expert, 16 * FR * WM at a time, against 16 * NF * WN weight rows (half of them the gate's, half the
// matching ones of the up projection with GLU): WM x WN wavefronts, each with FR x NF fragments of its own and all of
// k.
//
// One 16 x 16 x 64 step: lane (r, g), r = lane % 16, g = lane / 16, holds the codes 16g..16g+15 of row r of either
// side. Result register i is weight row 4g + i, input row r.
//
// Both sides go through LDS in stages of 128 bytes of a row, RING of them; a row's 16-byte pieces are swapped by its
// number (each lane fetches the piece that belongs where it writes) so that the lanes that LDS serves in a clock meet
// every bank once. Whole lines: four stages of 64 bytes are slower (2188 us for 2080 with the case of many rows below,
// 406 for 333 at 8 ranks x 32 tokens). The barrier comes when the current stage has been read, two fragments before its
// end; the next one's first fragments are read while those two multiply. The stage RING - 1 ahead is fetched between
// the next products (all at once behind the barrier the wavefronts stand still until the fetches are taken: 2021 us for
// 1937).
//
// Fragment f of wavefront row wm holds the tile's rows 16 * (f * WM + wm) and on, so that a tile with few rows leaves
// each wavefront as many: only those are fetched, read and multiplied (256 rows high, 2080 -> 2027 us; with 128 rows an
// expert 566 -> 491).
//
// What bounds it, with 64 experts of 7168 -> 4096 with SwiGLU or 256 of 2048 -> 7168. Few rows: the weights' bytes, 322
// us for 1.9 GB with 32 rows each (5.9 TB/s), 782 to 815 us for 4.2 GB in and out with 96 rows each. Many rows, skewed
// (1024 a rank, 8 ranks): 1721 to 1830 us, 2.1 to 2.2 POP/s, where the instruction alone reaches 4.2 on such values and
// 4.8 on constants. Power takes the clock to 1.6 GHz; of those cycles the matrix units are busy in 61 % and LDS reads
// in 26 %. Cut down (from 2080 us): 1475 without fetches, 1745 with fetches that hit the cache, 2086 without waiting
// for them, 1612 with the fetches alone; on zeros, which cost little power, 1835. So of what it takes beyond the instructions'
// own 917 us, about half is LDS reads, issue and their power (the loop without fetches), the other half the fetches' way
// through the caches and their energy, not their latency.
template <class T, int FR, int NF, int WM, int WN, int RING, bool GLU>
__global__ __launch_bounds__(WM *WN *kWave, WM *WN < 8 ? 1 : 2) void expert_product_kernel(ProductArgs a)
{
    constexpr int kThreads = WM * WN * kWave, kRowsW = WN * NF * 16, kRowsX = WM * FR * 16;
    constexpr int kSub = 2, kP = 4 * kSub;                    // steps, and 16-byte pieces of a row, in a stage
    constexpr int kLoadsW = kRowsW * kP / kThreads, kLoadsX = kRowsX * kP / kThreads;
    constexpr int kSizeW = kRowsW * kP, kSize = kSizeW + kRowsX * kP;
    constexpr int kBytes = kP * 16;                           // of a row in a stage
    static_assert(kRowsW * kP % kThreads == 0 && kRowsX * kP % kThreads == 0, "every thread carries as many pieces");
    static_assert(RING >= 2 && RING <= 4, "stages in LDS");
    // a stage's weights, then its inputs; an array a stage, so that the compiler tells them apart
    __shared__ u32x4 l0[kSize], l1[kSize], l2[RING > 2 ? kSize : 1], l3[RING > 3 ? kSize : 1];
    __shared__ float sw[kRowsW], sx[kRowsX];
    auto ring = [&](int i) -> u32x4 * { return i % RING == 0 ? l0 : (i % RING == 1 ? l1 : (i % RING == 2 ? l2 : l3)); };
    __shared__ Plan plan;
    const int total = make_plan<kRowsX, kThreads>(a, plan) * a.ntiles;
    const int tid = threadIdx.x, lane = tid % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), wm = wave / WN, wn = wave % WN;
    const int r = lane % 16, g = lane / 16;
    constexpr int kOut = GLU ? NF / 2 : NF, kOwn = NF * 16;   // output fragments and weight rows of a wavefront
    const int half = a.n / 2, stages = (a.k + kBytes - 1) / kBytes;
    // piece p of row q in LDS
    auto place = [](int q, int p) { return q * kP + (p ^ (q & 7)); };
    // a reader's pieces in each step: of fragment 0; the weights' others lie 16 rows apart, the inputs' 16 * WM (so
    // that a tile with few rows has as many for each wavefront)
    int wfrag[kSub], xfrag[kSub];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
        wfrag[u] = wn * kOwn * kP + place(r, 4 * u + g);
        xfrag[u] = kSizeW + wm * 16 * kP + place(r, 4 * u + g);
    }
    // the piece that this thread fetches of its rows (rows of its later pieces are a multiple of 8 on)
    const int piece = tid % kP ^ (tid / kP % 8);
    // Of the inputs' last stage this thread's piece may lie behind the row: an offset past the buffer then, which brings
    // zeros. (The weights' may too: of whatever comes there, times zeros.)
    const uint32_t behind = (stages - 1) * kBytes + 16 * piece < a.k ? 0u : 1u << 31;

    // Each XCD (workgroups go to the eight in turn) begins an eighth of the stages further on, and after the last one
    // comes the first: the sums are whole numbers, whose order does not matter, and the XCDs read different memory at a
    // time.
    const int turn = (int)(blockIdx.x % 8) * stages / 8;

    for (int t = blockIdx.x; t < total; t += gridDim.x) {
        const Tile tile = find_tile<kRowsX, kThreads>(a, plan, t / a.ntiles);
        const int tile0 = t % a.ntiles * (WN * kOut * 16);
        const uint8_t *wb = a.w + (size_t)tile.expert * a.n * a.k, *xb = a.x + (size_t)tile.row * a.k;
        const __amdgpu_buffer_rsrc_t wbuf = buffer_of(wb, (uint64_t)a.n * a.k);
        const int last = tile.end - 1 - tile.row;             // rows past the expert's last read the last one
        const __amdgpu_buffer_rsrc_t xbuf = buffer_of(xb, (uint64_t)(min(last, kRowsX - 1) + 1) * a.k);      // below 2^31
        // weight row of a place in the tile; columns past the last one read the last one's, and are not stored
        auto weight_row = [&](int q) -> uint32_t {
            const int c = GLU ? q / kOwn * (kOwn / 2) + q % (kOwn / 2) : q;
            return (GLU && q % kOwn >= kOwn / 2 ? half : 0) + min(tile0 + c, a.fo - 1);
        };
        uint32_t wo[kLoadsW], xo[kLoadsX];
#pragma unroll
        for (int i = 0; i < kLoadsW; ++i) wo[i] = weight_row((tid + i * kThreads) / kP) * a.k + 16 * piece;
#pragma unroll
        for (int i = 0; i < kLoadsX; ++i) xo[i] = (uint32_t)min((tid + i * kThreads) / kP, last) * a.k + 16 * piece;
        for (int q = tid; q < kRowsW; q += kThreads) sw[q] = a.ws[(size_t)tile.expert * a.n + weight_row(q)];
        for (int q = tid; q < kRowsX; q += kThreads) sx[q] = a.xs ? a.xs[tile.row + min(q, last)] : 1.f;

        i32x4 acc[FR][NF];
#pragma unroll
        for (int f = 0; f < FR; ++f)
#pragma unroll
            for (int j = 0; j < NF; ++j) acc[f][j] = i32x4{0, 0, 0, 0};
        // Fetches FROM..TO-1 of a whole stage's: the weights', then `loads` of the inputs'. Beyond the last stage the
        // last one is fetched again, and not used: a branch here would part the steps that it stands between, and the
        // waits count the fetches.
        auto fetch = [&](auto loads, int stage, int slot, int from, int to) {
            int at = min(stage, stages - 1) + turn;
            at -= at >= stages ? stages : 0;
            const uint32_t past = at == stages - 1 ? behind : 0u;
            u32x4 *wl = ring(slot), *xl = wl + kSizeW;
#pragma unroll
            for (int i = from; i < to; ++i) {
                if (i < kLoadsW)
                    fetch_lds(wbuf, wo[i], at * kBytes, wl + i * kThreads + wave * kWave);
                else if (i - kLoadsW < decltype(loads)::value)
                    fetch_lds(xbuf, xo[i - kLoadsW] | past, at * kBytes, xl + (i - kLoadsW) * kThreads + wave * kWave);
            }
        };
        u32x4 wf[2][NF], xf[2][FR];
        // fragments of step i, counted over the ring
        auto read_w = [&](int i) {
            const u32x4 *l = ring(i / kSub) + wfrag[i % kSub];
#pragma unroll
            for (int j = 0; j < NF; ++j) wf[i & 1][j] = l[j * 16 * kP];
        };
        auto read_x = [&](int i, int f) { xf[i & 1][f] = (ring(i / kSub) + xfrag[i % kSub])[f * WM * 16 * kP]; };
        auto multiply = [&](int i, int f) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
                acc[f][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, wf[i & 1][j]),
                                                                  __builtin_bit_cast(i32x4, xf[i & 1][f]), acc[f][j], 0, 0, 0);
        };
        // All stages, for the first LIVE fragments of every wavefront: the others have no rows.
        auto whole = [&](auto count) {
            constexpr int LIVE = decltype(count)::value, LAST = 2;
            using Loads = std::integral_constant<int, (kLoadsX * LIVE + FR - 1) / FR>;
            constexpr int kAll = kLoadsW + Loads::value, kLeft = (RING - 2) * kAll;
            static_assert(Loads::value * kThreads >= LIVE * WM * 16 * kP, "the rows of LIVE fragments are fetched");
#pragma unroll
            for (int i = 0; i < RING - 1; ++i) fetch(Loads(), i, i, 0, kAll);
            barrier_fetched<kLeft>();
            read_w(0);
#pragma unroll
            for (int f = 0; f < LAST; ++f) read_x(0, f);
            for (int s0 = 0; s0 < stages; s0 += RING) {
#pragma unroll
                for (int s = 0; s < RING; ++s) {
                    if (s0 + s >= stages) break;
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        const int i = s * kSub + u, next = (i + 1) % (RING * kSub);
#pragma unroll
                        for (int f = 0; f < LIVE - LAST; ++f) {
                            read_x(i, f + LAST);
                            multiply(i, f);
                            if (u == 0)
                                fetch(Loads(), s0 + s + RING - 1, (s + RING - 1) % RING, 2 * f,
                                      f == LIVE - LAST - 1 ? kAll : 2 * f + 2);
                            __builtin_amdgcn_sched_barrier(0);
                        }
                        if (LIVE == LAST && u == 0) fetch(Loads(), s0 + s + RING - 1, (s + RING - 1) % RING, 0, kAll);
                        if (u == kSub - 1) barrier_fetched<kLeft>();
                        read_w(next);
#pragma unroll
                        for (int f = 0; f < LAST; ++f) read_x(next, f);
                        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                        for (int f = LIVE - LAST; f < LIVE; ++f) multiply(i, f);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
        };
        const int live = last / (WM * 16) + 1;                // fragments that hold rows of the expert
        if constexpr (FR == 8) {
            if (live > 6) whole(std::integral_constant<int, 8>());
            else if (live > 4) whole(std::integral_constant<int, 6>());
            else if (live > 2) whole(std::integral_constant<int, 4>());
            else whole(std::integral_constant<int, 2>());
        } else {
            static_assert(FR == 2 || FR == 4, "the counts of fragments that the main loop is made for");
            if (FR > 2 && live > 2) whole(std::integral_constant<int, FR>());
            else whole(std::integral_constant<int, 2>());
        }
        barrier_fetched<0>();
        // Results leave by way of LDS, 16 rows of the wavefront's columns at a time, so that neighbouring lanes store
        // neighbouring 16 bytes
        constexpr int kPitch = kOut * 32 + 16;                // bytes; 16 more than the columns, to spread the banks
        constexpr int kLanes = kOut * 2;                      // lanes of a row
        static_assert(WM * WN * 16 * kPitch <= kSize * 16, "the wavefronts' rows fit into a stage");
        char *own = reinterpret_cast<char *>(l0) + wave * 16 * kPitch;
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            wave_fence();
            const float xs = sx[(f * WM + wm) * 16 + r];
#pragma unroll
            for (int j = 0; j < kOut; ++j) {
                float v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float *s = sw + wn * kOwn + j * 16 + 4 * g + i;
                    v[i] = product((float)acc[f][j][i] * s[0], xs);
                    if (GLU) v[i] = swiglu(v[i], (float)acc[f][j + kOut][i] * s[kOwn / 2] * xs);
                }
                u32x2 u;
                u[0] = (uint32_t)T::store(v[0]) | ((uint32_t)T::store(v[1]) << 16);
                u[1] = (uint32_t)T::store(v[2]) | ((uint32_t)T::store(v[3]) << 16);
                *reinterpret_cast<u32x2 *>(own + r * kPitch + j * 32 + g * 8) = u;
            }
            wave_fence();
#pragma unroll
            for (int i = 0; i < kOut * 32; i += kWave) {      // pieces of 16 bytes
                const int q = i + lane, row = tile.row + (f * WM + wm) * 16 + q / kLanes;
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

// Shapes of a tile: its rows and weight rows, the workgroups that run at once (two on a CU of the smallest), and what a
// round of them costs, in sixteenths of 128 x 256, whole or with 256 tiles at most (one on a CU). The large ones do most
// on what they fetch, the small ones fill the card where there are few, and pad few rows. (32 x 128 with four stages and
// one workgroup on a CU: 34.5 us with two tokens of the case above, 36.7 with three stages and two.)
struct TileShape {
    int rows, weights, threads, groups, cost, half, columns;     // columns: those of a row that it is worth while from
};
constexpr TileShape kShapes[] = {{128, 256, 512, 256, 16, 16, 0}, {256, 256, 512, 256, 24, 24, 0},
                                 {128, 128, 512, 256, 12, 12, 0}, {32, 128, 256, 256, 7, 7, 0}, {32, 64, 128, 512, 10, 6, 512}};

// The shape whose rounds cost least, the first of several, were the rows even over the experts (masked pairs' among
// them: no more is known here; an expert's last tile is half full). Measured over 200 products of 2 to 64 experts, 1 to 1000
// rows each, k 144 to 7168 and n 132 to 7168, half of them with SwiGLU, the choice costs 1.4 % over the best of the five in
// the mean and 30 % at most (128 x 128 for all of them 18 % in the mean). In us, for 256 x 256, 128 x 256, 128 x 128, 32 x
// 128 and 32 x 64, on inputs that change from pass to pass:
//    4 experts,   1 row each,  7168 -> 4096:    75   48   37   35   28
//    2 experts,  14 rows each, 3760 -> 3444:    55   40   24   23   15
//    2 experts, 250 rows each, 5376 -> 400:     51   32   21   15   14
//    8 experts, 250 rows each, 1152 -> 1600:    23   16   13   28   29
//   16 experts,  21 rows each, 6992 -> 268:     93   66   40   39   25
//   16 experts,  60 rows each, 7168 -> 4096:   101   87   88  116  122
//   16 experts, 250 rows each, 7168 -> 4096:   129  138  169  386  354
//   64 experts,   4 rows each, 7168 -> 4096:   357  312  314  310  312
//   64 experts, 250 rows each, 1152 -> 1600:    55   68   74  164  174
//   64 experts, 1000 rows each, 7168 -> 4096: 1685 1898 2335 4566 4210
int shape_of(int experts, int rows, int k, int out_columns, bool glu)
{
    const long long hit = std::max(1, std::min(experts, rows)), each = rows / hit;
    int best = 0;
    long long least = LLONG_MAX;
    for (int i = 0; i < (int)(sizeof kShapes / sizeof *kShapes); ++i) {
        const TileShape &s = kShapes[i];
        const int cols = s.weights / (glu ? 2 : 1);
        const long long high = hit * std::max<long long>(2 * s.rows, 2 * each + s.rows) / (2 * s.rows);
        const long long tiles = high * ((out_columns + cols - 1ll) / cols), rest = tiles % s.groups;
        const long long cost = tiles / s.groups * s.cost + (rest == 0 ? 0 : (rest <= 256 ? s.half : s.cost));
        if (k >= s.columns && cost < least) {
            least = cost;
            best = i;
        }
    }
    return best;
}

int check_rows(long long rows, int cols, int dtype)
{
    if (rows < 0 || cols < 1) return MOE_ERR_SHAPE;
    if (dtype != MOE_FP16 && dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_DTYPE;
    // a lane a piece: below 2^32 lanes; columns of a row's lanes are counted in 31 bits past its end
    if (rows > ((1ll << 31) - kRowThreads) / ((cols + kPiece - 1ll) / kPiece) || cols > 1 << 30) return MOE_ERR_SHAPE;
    return MOE_OK;
}

template <class F>
void by_type(int dtype, F f)
{
    if (dtype == MOE_FP16) f(F16());
    else if (dtype == MOE_BF16) f(BF16());
    else f(F32());
}

bool aligned_to(const void *p, int dtype) { return aligned(p, dtype == MOE_FP32 ? 4 : 2); }

RowsArgs rows_args(const void *in, void *out, long long rows, int cols)
{
    RowsArgs a;
    a.in = in;
    a.out = out;
    a.scales_in = nullptr;
    a.scales_out = nullptr;
    a.rows = rows;
    a.cols = cols;
    a.per_row = (cols + kPiece - 1) / kPiece;
    return a;
}

}  // namespace

extern "C" {

int moe_int8_quantize(const void *x, int64_t rows, int cols, int dtype, int8_t *codes, float *scales, void *stream)
{
    const int rc = check_rows(rows, cols, dtype);
    if (rc) return rc;
    if (rows == 0) return MOE_OK;
    if (!x || !codes || !scales) return MOE_ERR_NULLPTR;
    if (!aligned_to(x, dtype) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    RowsArgs a = rows_args(x, codes, rows, cols);
    a.scales_out = scales;
    // An input that fills the Infinity Cache passes it by: bf16 [32768, 7168] 115 us, 128 through it; a smaller one may
    // lie in it, fresh from the kernel before: [8192, 7168] 32 us past it, 28 through it.
    const bool once = rows * cols * (dtype == MOE_FP32 ? 4 : 2) >= kOnceBytes;
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) {
        using T = decltype(type);
        auto launch = [&](auto lanes, auto held) {
            constexpr int kLanes = decltype(lanes)::value, kRows = kRowThreads / kLanes;
            const dim3 g((unsigned)std::min<long long>((rows + kRows - 1) / kRows, 1 << 20));
            constexpr int kHeld = decltype(held)::value;
            if (once) hipLaunchKernelGGL((quantize_kernel<T, kLanes, kHeld, kHeld != 0>), g, dim3(kRowThreads), 0, st, a);
            else hipLaunchKernelGGL((quantize_kernel<T, kLanes, kHeld, false>), g, dim3(kRowThreads), 0, st, a);
        };
        using std::integral_constant;
        using Some = integral_constant<int, 16>;
        using Wave = integral_constant<int, kWave>;
        using All = integral_constant<int, kRowThreads>;
        const int p = a.per_row;
        if (p <= 16) launch(Some(), integral_constant<int, 1>());
        else if (p <= kWave) launch(Wave(), integral_constant<int, 1>());
        else if (p <= 2 * kWave) launch(Wave(), integral_constant<int, 2>());
        else if (p <= 4 * kWave) launch(Wave(), integral_constant<int, 4>());
        else if (p <= 2 * kRowThreads) launch(All(), integral_constant<int, 2>());
        else if (p <= 4 * kRowThreads) launch(All(), integral_constant<int, 4>());
        else launch(All(), integral_constant<int, 0>());
    });
    return launched();
}

int moe_int8_dequantize(const int8_t *codes, const float *scales, int64_t rows, int cols, int dtype, void *out, void *stream)
{
    const int rc = check_rows(rows, cols, dtype);
    if (rc) return rc;
    if (rows == 0) return MOE_OK;
    if (!codes || !scales || !out) return MOE_ERR_NULLPTR;
    if (!aligned_to(out, dtype) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
    RowsArgs a = rows_args(codes, out, rows, cols);
    a.scales_in = scales;
    const dim3 g((unsigned)((rows * a.per_row + kRowThreads - 1) / kRowThreads)), b(kRowThreads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) { hipLaunchKernelGGL(dequantize_kernel<decltype(type)>, g, b, 0, st, a); });
    return launched();
}

int moe_expert_product_int8(const int8_t *x, const float *x_scales, const int8_t *weights, const float *weight_scales,
                            const int32_t *ep_recv_count, int ep_world, int experts_per_rank, int rows, int k, int n,
                            int activation, int dtype, void *out, void *stream)
{
    if (ep_world < kMinWorld || ep_world > kMaxWorld || experts_per_rank < 1 ||
        (long long)ep_world * experts_per_rank > kMaxExperts || rows < 0 || k < kPiece || k % kPiece || n < 1)
        return MOE_ERR_SHAPE;
    if (dtype != MOE_FP16 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
    if (activation != MOE_ACT_NONE && activation != MOE_ACT_SWIGLU) return MOE_ERR_SHAPE;
    const bool glu = activation == MOE_ACT_SWIGLU;
    if (glu && n % 2) return MOE_ERR_SHAPE;
    // sums of k products of at most 2^14 stay below 2^31; offsets inside one expert's weights in 31 bits
    if (k > (INT_MAX >> 14) || (long long)n * k > 1ll << 31) return MOE_ERR_SHAPE;
    ProductArgs a;
    a.W = ep_world;
    a.epr = experts_per_rank;
    a.E = ep_world * experts_per_rank;
    a.S = a.E;                                  // segments of a rank: experts_per_rank * ep_world
    a.rows = rows;
    a.k = k;
    a.n = n;
    a.fo = glu ? n / 2 : n;
    const int shape = shape_of(a.E, rows, k, a.fo, glu);
    const TileShape &tile = kShapes[shape];
    const int cols = tile.weights / (glu ? 2 : 1), groups = tile.groups;
    a.ntiles = (int)((a.fo + cols - 1ll) / cols);
    // a tile starts at every expert's first row, so at most this many
    const long long mtiles = rows / tile.rows + std::min(a.E, rows);
    // rows and tiles are counted past the last one by up to a tile's height and a stride of the grid
    if (rows > INT_MAX - 256 || mtiles * a.ntiles > INT_MAX - groups) return MOE_ERR_SHAPE;
    if (rows == 0) return MOE_OK;
    if (!x || !weights || !weight_scales || !ep_recv_count || !out) return MOE_ERR_NULLPTR;
    if (!aligned(x, 16) || !aligned(weights, 16) || !aligned(x_scales, 4) || !aligned(weight_scales, 4) ||
        !aligned(ep_recv_count, 4) || !aligned(out, 2))
        return MOE_ERR_ALIGN;
    a.x = reinterpret_cast<const uint8_t *>(x);
    a.w = reinterpret_cast<const uint8_t *>(weights);
    a.xs = x_scales;
    a.ws = weight_scales;
    a.erc = ep_recv_count;
    a.out = out;
    const dim3 g((unsigned)std::min<long long>(mtiles * a.ntiles, groups)), b(tile.threads);
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    auto launch = [&](auto type, auto act) {
        using T = decltype(type);
        constexpr bool kGlu = decltype(act)::value;
        if (shape == 0) hipLaunchKernelGGL((expert_product_kernel<T, 4, 4, 2, 4, 3, kGlu>), g, b, 0, st, a);
        else if (shape == 1) hipLaunchKernelGGL((expert_product_kernel<T, 8, 4, 2, 4, 2, kGlu>), g, b, 0, st, a);
        else if (shape == 2) hipLaunchKernelGGL((expert_product_kernel<T, 4, 2, 2, 4, 4, kGlu>), g, b, 0, st, a);
        else if (shape == 3) hipLaunchKernelGGL((expert_product_kernel<T, 2, 2, 1, 4, 4, kGlu>), g, b, 0, st, a);
        else hipLaunchKernelGGL((expert_product_kernel<T, 2, 2, 1, 2, 4, kGlu>), g, b, 0, st, a);
    };
    if (dtype == MOE_FP16 && glu) launch(F16(), std::true_type());
    else if (dtype == MOE_FP16) launch(F16(), std::false_type());
    else if (glu) launch(BF16(), std::true_type());
    else launch(BF16(), std::false_type());
    return launched();
}

}  // extern "C"
