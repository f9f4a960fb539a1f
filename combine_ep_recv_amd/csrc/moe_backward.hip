// moe_backward.hip -- the gradients of combine and dispatch (gfx950, wave64).
//
// With g the gradient of x_out, y the experts' rows and w the weights (row(t, k) is the row that dispatch gave to pair
// (t, k)):
//   combine   grad_y[row(t, k)] = w[t, k] * g[t]
//             grad_w[t, k] = sum over the columns of y[row(t, k)] * g[t]; 0 for a pair without a row, except that a copy
//             expert's row is ori_x[t] and const expert j's const_x[j]
//             grad_ori_x[t] = (sum over copy pairs of w[t, k]) * g[t]
//             grad_const_x[j] = sum over const expert j's pairs of w[t, k] * g[t]
//   dispatch  grad_x[t] = add[t] + sum over k of grad_expand_x[row(t, k)]
// Everything is held in fp32 and rounded once, and every sum has a fixed order.

#include "moe_types.h"

#include <limits.h>

#include <algorithm>
#include <type_traits>

namespace {

using namespace moe_detail;

constexpr long long kMaxTokens = (1ll << 24) - 1;
constexpr int kPiece = 8;                  // elements of 16 bytes
// Threads of a workgroup, by the columns alone, so that a sum's order goes by them alone: one wavefront up to so many,
// four above. 8 ranks x 1024 tokens, 512 columns: combine's gradient 27.0 us, dispatch's 17.9, with four 46.6 and 23.0;
// 16 x 256, 1024 columns 23.7 and 15.1, 29.7 and 16.6; 4 x 515, 2048 columns 20.6 and 13.5, 22.5 and 15.2; 16 x 256,
// 7168 columns 193 and 104, 203 and 100, but 8 x 32 24.7 and 9.5, 16.9 and 8.8.
constexpr int kNarrow = 64, kWide = 256, kNarrowCols = 2048;
int threads_of(int h) { return h <= kNarrowCols ? kNarrow : kWide; }
// Rows that fill the Infinity Cache pass the caches by: 16 ranks x 256 tokens, top-8, bf16 rows of 7168, combine's
// gradient 203 us and dispatch's 100, 217 and 106 through them; smaller ones may lie in them, fresh from the experts: 8
// ranks x 32 tokens 15.4 and 7.9 us through them, 16.9 and 8.8 past them.
constexpr long long kOnceBytes = 256ll << 20;
// Up to so many pairs combine's gradient gives each pair a workgroup of its own: 1024 pairs (8 ranks x 16 tokens, 7168)
// 9.4 us, 9.8 with a workgroup a token; 2048 14.9 and 12.9, 8192 51 and 38.5.
constexpr long long kFewPairs = 1024;
// Up to so many tokens dispatch's gradient parts their rows: 128 tokens of 7168 4.4 us, 6.9 in one piece; 256 7.8 and
// 8.6, 512 13.4 and 12.8.
constexpr long long kFewTokens = 256;
constexpr int kNone = -1, kCopy = -2, kConst = -3;      // a pair without a row, of a copy expert, of const expert kConst - j

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));      // rows start at any element

struct Routing {
    const int32_t *assist, *erc, *ids;
    const uint8_t *mask;
    int mask_kind;
    int W, bs, K, epr, E, S, R;
    int zero_end, copy_end, const_end;     // special ids: [zero_end, copy_end) copy, [copy_end, const_end) const
};

// Tokens' rows in LDS: where each rank's rows begin, and the row (or kNone, kCopy, kConst - j) of each of a token's
// pairs.
struct Rows {
    uint32_t before[kMaxWorld];
    int row[kMaxExperts];
};

// Finds the rows of token t's pairs: pair (t, k) lies in segment (local expert, source rank) of its expert's rank,
// whose rows are in order of their tokens, so that assist_info's token column is searched by halves. (No pass over all
// rows first, as combine's slots, which would be a launch more: a segment has few rows, and the loads hit the L2. All
// 64 lanes looking at a segment at once were no faster: 14.7 us for 15.3 at 8 ranks x 32 tokens, 12.7 for 11.4 at 4 x
// 515.) The first wavefront calls it; the caller puts a barrier behind it. Whatever the arrays hold, rows stay in [0,
// R).
__device__ __forceinline__ void find_rows(const Routing &a, int t, Rows &rows)
{
    const int lane = threadIdx.x;
    const int s = t / a.bs, tok = t - s * a.bs;
    uint32_t carry = 0;
    for (int q = 0; q < a.W; q += kWave) {
        const int rank = q + lane;
        const int total = rank < a.W ? a.erc[(size_t)rank * a.S + a.S - 1] : 0;
        const uint32_t inc = min((uint32_t)a.R, wave_scan((uint32_t)min(max(total, 0), a.R), (uint32_t)a.R) + carry);
        // the sums before this rank: one lane up
        const uint32_t before = (uint32_t)__builtin_amdgcn_update_dpp((int)carry, (int)inc, 0x138, 0xf, 0xf, false);
        if (rank < a.W) rows.before[rank] = before;
        carry = (uint32_t)__builtin_amdgcn_readlane((int)inc, kWave - 1);
    }
    wave_fence();
    for (int k = lane; k < a.K; k += kWave) {
        const size_t p = (size_t)t * a.K + k;
        const int e = a.ids[p];
        bool on = true;
        if (a.mask_kind != MOE_MASK_NONE) on = a.mask[a.mask_kind == MOE_MASK_TOKEN ? (size_t)t : p] != 0;
        int row = kNone;
        if (on && (unsigned)e < (unsigned)a.E) {
            const int r = e / a.epr, seg = (e - r * a.epr) * a.W + s;
            const int32_t *c = a.erc + (size_t)r * a.S + seg;
            const uint32_t base = rows.before[r];
            uint32_t lo = seg ? (uint32_t)min(max(c[-1], 0), a.R) : 0u, hi = (uint32_t)min(max(c[0], 0), a.R);
            lo = min((uint32_t)a.R, base + lo);
            hi = min((uint32_t)a.R, base + hi);
            const uint32_t end = hi;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) >> 1;
                if (a.assist[(size_t)mid * 3 + 1] < tok) lo = mid + 1;
                else hi = mid;
            }
            if (lo < end && a.assist[(size_t)lo * 3 + 1] == tok) row = (int)lo;
        } else if (on && e >= a.zero_end && e < a.const_end) {
            row = e < a.copy_end ? kCopy : kConst - (e - a.copy_end);
        }
        rows.row[k] = row;
    }
}

// 16 bytes of a row; ONCE: past the caches
template <bool ONCE>
__device__ __forceinline__ u32x4 load16(const void *p)
{
    const u32x4_a2 *q = static_cast<const u32x4_a2 *>(p);
    return ONCE ? __builtin_nontemporal_load(q) : *q;
}
__device__ __forceinline__ void store16(void *p, u32x4 v)
{
    __builtin_nontemporal_store(v, static_cast<u32x4_a2 *>(p));
}
template <class T>
__device__ __forceinline__ void unpack(u32x4 v, float (&x)[kPiece])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = T::load((uint16_t)(v[i] & 0xffff));
        x[2 * i + 1] = T::load((uint16_t)(v[i] >> 16));
    }
}
template <class T>
__device__ __forceinline__ u32x4 pack(const float (&x)[kPiece])
{
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (uint32_t)T::store(x[2 * i]) | ((uint32_t)T::store(x[2 * i + 1]) << 16);
    return v;
}

// --------------------------------------------------------------------------
// combine
// --------------------------------------------------------------------------

// The const experts' table: every pair adds to one row of it. A workgroup takes expert j, a slice of columns and a part
// of the tokens: it lists the part's pairs of expert j in order, then adds their rows, and a second kernel joins the
// parts. These workgroups come first in combine's launch (a launch of their own is 8 us more with 4 ranks of 515
// tokens).
constexpr int kMostSplits = 64, kSplitTokens = 32, kAhead = 8;
// Tokens of a part that are added by themselves, before their sum goes to the part's: a part has up to 2^18 tokens, and
// fp32 sums of so many like terms one after the other are off by 0.35 % (seven half steps of fp16), by 0.01 % so.
constexpr int kBlockTokens = 1024;

struct ConstArgs {
    const uint16_t *grad;
    const float *w;
    const int32_t *ids;
    const uint8_t *mask;
    float *sums;                           // [const experts, splits, h], or NULL where one part is all
    uint16_t *out;
    int mask_kind, N, K, h, first_id, slices, splits, per, join_slices;
};

template <int THREADS>
struct ConstList {
    int pair[4 * THREADS];                 // of as many looked at between two lists
    int count[4][THREADS / kWave];
};

template <class T, int THREADS>
__device__ __forceinline__ void const_backward(const ConstArgs &a, int block, ConstList<THREADS> &found)
{
    constexpr int kWaves = THREADS / kWave, kScan = 4 * THREADS;
    int(&list)[kScan] = found.pair;
    int(&count)[4][kWaves] = found.count;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int j = block / (a.slices * a.splits), q = block - j * (a.slices * a.splits);
    const int split = q / a.slices;
    const long long at = (long long)(q - split * a.slices) * (THREADS * kPiece) + tid * kPiece;
    const int id = a.first_id + j;
    // columns of this lane, the last eight where it has fewer (those of its neighbour among them, which both store)
    const int live = at >= a.h ? 0 : min(a.h, kPiece);
    const long long col = max(min(at, (long long)a.h - kPiece), 0ll);
    const long long from = (long long)split * a.per * a.K, to = min((long long)a.N, (long long)(split + 1) * a.per) * a.K;
    float acc[kPiece], sum[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) acc[i] = sum[i] = 0.f;
    static_assert(kBlockTokens % kScan == 0, "lists end where blocks do");
    int left = kBlockTokens * a.K;
    for (long long base = from; base < to; base += kScan) {
        uint64_t hit[4];
        bool mine[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long p = base + u * THREADS + tid;
            mine[u] = p < to && a.ids[p] == id;
            if (mine[u] && a.mask_kind != MOE_MASK_NONE)
                mine[u] = a.mask[a.mask_kind == MOE_MASK_TOKEN ? p / a.K : p] != 0;
            hit[u] = __builtin_amdgcn_ballot_w64(mine[u]);
            if (lane == 0) count[u][wave] = __popcll(hit[u]);
        }
        __syncthreads();
        int total = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            int at = total;
#pragma unroll
            for (int i = 0; i < kWaves; ++i) {
                if (i < wave) at += count[u][i];
                total += count[u][i];
            }
            if (mine[u]) list[at + __popcll(hit[u] & ((1ull << lane) - 1))] = (int)(base + u * THREADS + tid);
        }
        __syncthreads();
        // kAhead rows on their way at a time; the list's last pair stands in for those past its end
        for (int i = 0; i < total; i += kAhead) {
            const uint16_t *g[kAhead];
            float w[kAhead];
#pragma unroll
            for (int q = 0; q < kAhead; ++q) {
                const int p = __builtin_amdgcn_readfirstlane(list[min(i + q, total - 1)]);
                g[q] = a.grad + (size_t)(p / a.K) * a.h + col;
                w[q] = a.w[p];
            }
            if (live == kPiece) {
                u32x4 v[kAhead];
#pragma unroll
                for (int q = 0; q < kAhead; ++q) v[q] = *reinterpret_cast<const u32x4_a2 *>(g[q]);
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    if (i + q >= total) break;
                    float x[kPiece];
                    unpack<T>(v[q], x);
#pragma unroll
                    for (int c = 0; c < kPiece; ++c) acc[c] = __builtin_fmaf(w[q], x[c], acc[c]);
                }
            } else {
#pragma unroll
                for (int q = 0; q < kAhead; ++q) {
                    if (i + q >= total) break;
#pragma unroll
                    for (int c = 0; c < kPiece; ++c)
                        if (c < live) acc[c] = __builtin_fmaf(w[q], T::load(g[q][c]), acc[c]);
                }
            }
        }
        left -= kScan;
        if (left == 0 || base + kScan >= to) {
#pragma unroll
            for (int c = 0; c < kPiece; ++c) {
                sum[c] += acc[c];
                acc[c] = 0.f;
            }
            left = kBlockTokens * a.K;
        }
        __syncthreads();
    }
#pragma unroll
    for (int c = 0; c < kPiece; ++c) {
        if (c >= live) continue;
        if (a.sums) a.sums[((size_t)j * a.splits + split) * a.h + col + c] = sum[c];
        else a.out[(size_t)j * a.h + col + c] = T::store(sum[c]);
    }
}

struct CombineBackwardArgs {
    Routing r;
    const uint16_t *grad, *y, *ori_x, *const_x;
    const float *w;
    uint16_t *grad_y, *grad_ori;
    float *grad_w;
    int h, parts;
    ConstArgs table;
    int table_blocks;                      // workgroups of the const experts' gradient, before the tokens'
};

// A workgroup takes token t and every `parts`th block of KB of its pairs: g[t] is read once for KB rows, which are read
// and written once. Rows in pieces of 16 bytes a lane (at any alignment), the h % 8 last elements one a lane. Each lane
// adds the products of its own columns, eight neighbours in order and then those 8 * THREADS on; a wavefront's lanes
// and then the wavefronts are joined in a fixed order, the same for every KB.
//
// Memory bounds it: 3 operations an element of 4 bytes. 16 ranks x 256 tokens, top-8, bf16 rows of 7168: 1.0 GB in 197
// to 203 us, 4.9 to 5.1 TB/s, where a large copy reaches 5.2.
template <class T, int KB, bool ONCE, bool TABLE, int THREADS>
__global__ __launch_bounds__(THREADS) void combine_backward_kernel(CombineBackwardArgs a)
{
    constexpr int kWaves = THREADS / kWave;
    __shared__ Rows rows;
    __shared__ float part[kWaves][KB];
    int block = blockIdx.x;
    if constexpr (TABLE) {
        __shared__ ConstList<THREADS> found;
        if (block < a.table_blocks) return const_backward<T, THREADS>(a.table, block, found);
        block -= a.table_blocks;
    }
    const int t = block / a.parts, first = block - t * a.parts;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int K = a.r.K, pieces = a.h / kPiece, tail = a.h - pieces * kPiece, rest = pieces * kPiece + min(tid, tail);
    if (wave == 0) find_rows(a.r, t, rows);
    __syncthreads();
    const uint16_t *g = a.grad + (size_t)t * a.h;
    for (int kb = first * KB; kb < K; kb += a.parts * KB) {
        const uint16_t *src[KB];
        int row[KB];
        float w[KB], acc[KB];
#pragma unroll
        for (int i = 0; i < KB; ++i) {
            row[i] = __builtin_amdgcn_readfirstlane(kb + i < K ? rows.row[kb + i] : kNone);
            w[i] = kb + i < K ? a.w[(size_t)t * K + kb + i] : 0.f;
            // a pair without a row reads the gradient's again, which is in the cache: a load that hangs on the pair
            // would have the others waited for
            src[i] = row[i] >= 0       ? a.y + (size_t)row[i] * a.h
                     : row[i] == kNone ? g
                     : row[i] == kCopy ? a.ori_x + (size_t)t * a.h
                                       : a.const_x + (size_t)(kConst - row[i]) * a.h;
            acc[i] = 0.f;
        }
        for (int c = tid; c < pieces; c += THREADS) {
            u32x4 v[KB];
            const u32x4 gv = *reinterpret_cast<const u32x4_a2 *>(g + c * kPiece);
#pragma unroll
            for (int i = 0; i < KB; ++i)
                v[i] = load16<ONCE>(src[i] + c * kPiece);
            float gx[kPiece];
            unpack<T>(gv, gx);
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                float x[kPiece], o[kPiece];
                unpack<T>(v[i], x);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) {
                    acc[i] = __builtin_fmaf(x[j], gx[j], acc[i]);
                    o[j] = product(w[i], gx[j]);
                }
                if (row[i] >= 0) store16(a.grad_y + (size_t)row[i] * a.h + c * kPiece, pack<T>(o));
            }
        }
        if (tid < tail) {
            const float gx = T::load(g[rest]);
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                acc[i] = __builtin_fmaf(T::load(src[i][rest]), gx, acc[i]);
                if (row[i] >= 0) a.grad_y[(size_t)row[i] * a.h + rest] = T::store(product(w[i], gx));
            }
        }
#pragma unroll
        for (int i = 0; i < KB; ++i) {
            const float v = wave_sum(acc[i]);
            if (lane == 0) part[wave][i] = v;
        }
        __syncthreads();
        if (tid < KB && kb + tid < K) {
            float v = part[0][tid];
#pragma unroll
            for (int i = 1; i < kWaves; ++i) v += part[i][tid];
            a.grad_w[(size_t)t * K + kb + tid] = rows.row[kb + tid] == kNone ? 0.f : v;
        }
        __syncthreads();
    }
    if (a.grad_ori && first == 0) {
        // a token without copy pairs gets 0 whatever its gradient holds
        float w = 0.f;
        bool mine = false;
        for (int k = lane; k < K; k += kWave)
            if (rows.row[k] == kCopy) {
                w += a.w[(size_t)t * K + k];
                mine = true;
            }
        w = wave_sum(w);
        const bool some = __builtin_amdgcn_ballot_w64(mine) != 0;
        uint16_t *o = a.grad_ori + (size_t)t * a.h;
        for (int c = tid; c < pieces; c += THREADS) {
            float x[kPiece];
            unpack<T>(*reinterpret_cast<const u32x4_a2 *>(g + c * kPiece), x);
#pragma unroll
            for (int j = 0; j < kPiece; ++j) x[j] = some ? product(w, x[j]) : 0.f;
            store16(o + c * kPiece, pack<T>(x));
        }
        if (tid < tail) o[rest] = T::store(some ? product(w, T::load(g[rest])) : 0.f);
    }
}

template <class T>
__global__ __launch_bounds__(kWide) void const_join_kernel(ConstArgs a)
{
    const int j = blockIdx.x / a.join_slices;
    const long long col = (long long)(blockIdx.x - j * a.join_slices) * kWide + threadIdx.x;
    if (col >= a.h) return;
    float v = 0.f;
#pragma unroll 8
    for (int i = 0; i < a.splits; ++i) v += a.sums[((size_t)j * a.splits + i) * a.h + col];
    a.out[(size_t)j * a.h + col] = T::store(v);
}

// --------------------------------------------------------------------------
// dispatch
// --------------------------------------------------------------------------

struct DispatchBackwardArgs {
    Routing r;
    const uint16_t *grad, *add;
    const float *grad_scales_in;
    uint16_t *out;
    float *grad_scales;
    int h, slices;
};

// A workgroup takes token t and every `slices`th THREADS pieces of its row, eight rows' pieces on their way at a time.
// Memory bounds it: 529 MB in 97 to 100 us (5.3 TB/s) at 16 ranks x 256 tokens, top-8, bf16 rows of 7168.
template <class T, bool ONCE, int THREADS>
__global__ __launch_bounds__(THREADS) void dispatch_backward_kernel(DispatchBackwardArgs a)
{
    __shared__ Rows rows;
    const int t = blockIdx.x / a.slices, slice = blockIdx.x - t * a.slices;
    const int tid = threadIdx.x, K = a.r.K, pieces = a.h / kPiece, tail = a.h - pieces * kPiece;
    if (tid < kWave) find_rows(a.r, t, rows);
    __syncthreads();
    constexpr int KB = 8;
    for (int c = slice * THREADS + tid; c < pieces; c += a.slices * THREADS) {
        float acc[kPiece];
        u32x4 v[KB];
        if (a.add) {
            unpack<T>(load16<ONCE>(a.add + (size_t)t * a.h + c * kPiece), acc);
        } else {
#pragma unroll
            for (int i = 0; i < kPiece; ++i) acc[i] = 0.f;
        }
        for (int kb = 0; kb < K; kb += KB) {
            int row[KB];
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                row[i] = __builtin_amdgcn_readfirstlane(kb + i < K ? rows.row[kb + i] : kNone);
                v[i] = load16<ONCE>(a.grad + (size_t)max(row[i], 0) * a.h + c * kPiece);        // without a row: see above
            }
#pragma unroll
            for (int i = 0; i < KB; ++i) {
                if (row[i] < 0) continue;
                float x[kPiece];
                unpack<T>(v[i], x);
#pragma unroll
                for (int j = 0; j < kPiece; ++j) acc[j] += x[j];
            }
        }
        store16(a.out + (size_t)t * a.h + c * kPiece, pack<T>(acc));
    }
    if (slice == 0 && tid < tail) {
        const int rest = pieces * kPiece + tid;
        float v = a.add ? T::load(a.add[(size_t)t * a.h + rest]) : 0.f;
        for (int k = 0; k < K; ++k)
            if (rows.row[k] >= 0) v += T::load(a.grad[(size_t)rows.row[k] * a.h + rest]);
        a.out[(size_t)t * a.h + rest] = T::store(v);
    }
    if (slice == 0 && a.grad_scales)
        for (int k = tid; k < K; k += THREADS)
            a.grad_scales[(size_t)t * K + k] = rows.row[k] >= 0 ? a.grad_scales_in[rows.row[k]] : 0.f;
}

// --------------------------------------------------------------------------
// host side
// --------------------------------------------------------------------------

int check_call(int W, int bs, int epr, int h, int K, int dtype)
{
    if (dtype != MOE_FP16 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
    if (W < kMinWorld || W > kMaxWorld || epr < 1 || bs < 0 || h < 1 || K < 1) return MOE_ERR_SHAPE;
    const long long E = (long long)W * epr, N = (long long)W * bs;
    if (E > kMaxExperts || K > E || N > kMaxTokens || N * K > INT_MAX) return MOE_ERR_SHAPE;
    // dispatch's bound on a token's slices of 128 elements
    if (N * ((h + 127ll) / 128) >= 1ll << 25) return MOE_ERR_SHAPE;
    return MOE_OK;
}

int check_mask(const uint8_t *mask, int kind, long long N)
{
    if (kind < MOE_MASK_NONE || kind > MOE_MASK_PAIR) return MOE_ERR_MASK;
    if ((kind != MOE_MASK_NONE) != (mask != nullptr) && N > 0) return MOE_ERR_MASK;
    return kind == MOE_MASK_NONE && mask ? MOE_ERR_MASK : MOE_OK;
}

Routing routing_of(const int32_t *assist, const int32_t *erc, const int32_t *ids, const uint8_t *mask, int mask_kind, int W,
                   int bs, int epr, int K)
{
    Routing r;
    r.assist = assist;
    r.erc = erc;
    r.ids = ids;
    r.mask = mask;
    r.mask_kind = mask_kind;
    r.W = W;
    r.bs = bs;
    r.K = K;
    r.epr = epr;
    r.E = r.S = W * epr;
    r.R = (int)((long long)W * bs * K);
    r.zero_end = r.copy_end = r.const_end = r.E;
    return r;
}

// f(element type, whether rows of this many bytes pass the caches by, threads of a workgroup for h columns)
template <class F>
void by_type(int dtype, long long bytes, int h, F f)
{
    auto sized = [&](auto type) {
        const bool once = bytes >= kOnceBytes, narrow = threads_of(h) == kNarrow;
        using Narrow = std::integral_constant<int, kNarrow>;
        using Wide = std::integral_constant<int, kWide>;
        if (once && narrow) f(type, std::true_type(), Narrow());
        else if (once) f(type, std::true_type(), Wide());
        else if (narrow) f(type, std::false_type(), Narrow());
        else f(type, std::false_type(), Wide());
    };
    if (dtype == MOE_FP16) sized(F16());
    else sized(BF16());
}

// Parts of the tokens for the const experts' sums: by the tokens alone, so that a sum's order does not change with h.
int splits_of(long long N) { return (int)std::min<long long>(kMostSplits, (N + kSplitTokens - 1) / kSplitTokens); }

}  // namespace

extern "C" {

int moe_combine_backward_workspace_size(int ep_world, int bs, int experts_per_rank, int h, int topk, int dtype,
                                        int const_expert_num, size_t *bytes)
{
    if (!bytes) return MOE_ERR_NULLPTR;
    const int rc = check_call(ep_world, bs, experts_per_rank, h, topk, dtype);
    if (rc) return rc;
    const int splits = splits_of((long long)ep_world * bs);
    // a launch has fewer than 2^24 workgroups, the tokens' among them
    const long long cols = threads_of(h) * kPiece;
    const long long slices = std::max((h + cols - 1) / cols * std::max(splits, 1), (h + kWide - 1ll) / kWide);
    const long long tokens = std::max((long long)ep_world * bs, kFewPairs);
    if (const_expert_num < 0 || (const_expert_num > 0 && const_expert_num * slices + tokens >= 1ll << 24)) return MOE_ERR_SHAPE;
    *bytes = splits > 1 ? (size_t)const_expert_num * splits * h * sizeof(float) : 0;
    return MOE_OK;
}

int moe_combine_backward(const void *grad_out, const void *expand_x, const int32_t *assist_info, const int32_t *ep_recv_count,
                         const int32_t *expert_ids, const float *expert_scales, const uint8_t *x_active_mask, int mask_kind,
                         const moe_special_experts *special, int ep_world, int bs, int experts_per_rank, int h, int topk,
                         int dtype, void *grad_expand_x, float *grad_scales, void *grad_ori_x, void *grad_const_x,
                         void *workspace, size_t workspace_bytes, void *stream)
{
    const int zero_n = special ? special->zero_expert_num : 0, copy_n = special ? special->copy_expert_num : 0;
    const int const_n = special ? special->const_expert_num : 0;
    size_t need = 0;
    int rc = check_call(ep_world, bs, experts_per_rank, h, topk, dtype);
    if (rc) return rc;
    if (zero_n < 0 || copy_n < 0 || const_n < 0) return MOE_ERR_SHAPE;
    const long long N = (long long)ep_world * bs, E = (long long)ep_world * experts_per_rank;
    if (E + zero_n + copy_n + const_n > INT_MAX) return MOE_ERR_SHAPE;
    const int table = const_n > 0 && grad_const_x ? const_n : 0;
    if ((rc = moe_combine_backward_workspace_size(ep_world, bs, experts_per_rank, h, topk, dtype, table, &need))) return rc;
    if (!ep_recv_count) return MOE_ERR_NULLPTR;
    if (N > 0 && (!grad_out || !expand_x || !assist_info || !expert_ids || !expert_scales || !grad_expand_x || !grad_scales))
        return MOE_ERR_NULLPTR;
    if ((rc = check_mask(x_active_mask, mask_kind, N))) return rc;
    const void *ori_x = copy_n > 0 ? special->ori_x : nullptr, *const_x = const_n > 0 ? special->const_x : nullptr;
    if (N > 0 && ((copy_n > 0 && !ori_x) || (const_n > 0 && !const_x))) return MOE_ERR_NULLPTR;
    if ((grad_ori_x && copy_n == 0) || (grad_const_x && const_n == 0)) return MOE_ERR_NULLPTR;
    if (need > 0 && !workspace) return MOE_ERR_NULLPTR;
    if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(grad_out, 2) || !aligned(expand_x, 2) || !aligned(assist_info, 4) || !aligned(ep_recv_count, 4) ||
        !aligned(expert_ids, 4) || !aligned(expert_scales, 4) || !aligned(grad_expand_x, 2) || !aligned(grad_scales, 4) ||
        !aligned(ori_x, 2) || !aligned(const_x, 2) || !aligned(grad_ori_x, 2) || !aligned(grad_const_x, 2) ||
        (need > 0 && !aligned(workspace, 16)))
        return MOE_ERR_ALIGN;
    if (N == 0 && table == 0) return MOE_OK;
    CombineBackwardArgs a;
    a.r = routing_of(assist_info, ep_recv_count, expert_ids, x_active_mask, mask_kind, ep_world, bs, experts_per_rank, topk);
    a.r.zero_end = a.r.E + zero_n;
    a.r.copy_end = a.r.zero_end + copy_n;
    a.r.const_end = a.r.copy_end + const_n;
    a.grad = static_cast<const uint16_t *>(grad_out);
    a.y = static_cast<const uint16_t *>(expand_x);
    a.ori_x = static_cast<const uint16_t *>(ori_x);
    a.const_x = static_cast<const uint16_t *>(const_x);
    a.w = expert_scales;
    a.grad_y = static_cast<uint16_t *>(grad_expand_x);
    a.grad_ori = static_cast<uint16_t *>(grad_ori_x);
    a.grad_w = grad_scales;
    a.h = h;
    // few pairs: a workgroup each, one token's eight at a time otherwise
    const bool few = N * topk <= kFewPairs;
    a.parts = few ? topk : 1;
    ConstArgs &c = a.table;
    c.grad = a.grad;
    c.w = expert_scales;
    c.ids = expert_ids;
    c.mask = x_active_mask;
    c.mask_kind = mask_kind;
    c.N = (int)N;
    c.K = topk;
    c.h = h;
    c.first_id = a.r.copy_end;
    c.splits = std::max(1, splits_of(N));
    c.per = (int)((N + c.splits - 1) / c.splits);
    const long long cols = threads_of(h) * kPiece;          // of a workgroup at a time
    c.slices = (int)((h + cols - 1) / cols);
    c.join_slices = (int)((h + kWide - 1ll) / kWide);
    c.sums = c.splits > 1 ? static_cast<float *>(workspace) : nullptr;
    c.out = static_cast<uint16_t *>(grad_const_x);
    a.table_blocks = table * c.slices * c.splits;
    const dim3 g((unsigned)(a.table_blocks + N * a.parts));
    const dim3 join((unsigned)(table * c.join_slices));
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, N * topk * h * 2, h, [&](auto type, auto once, auto threads) {
        using T = decltype(type);
        constexpr bool kOnce = decltype(once)::value;
        constexpr int kT = decltype(threads)::value;
        const dim3 b(kT);
        if (few && table) hipLaunchKernelGGL((combine_backward_kernel<T, 1, kOnce, true, kT>), g, b, 0, st, a);
        else if (few) hipLaunchKernelGGL((combine_backward_kernel<T, 1, kOnce, false, kT>), g, b, 0, st, a);
        else if (table) hipLaunchKernelGGL((combine_backward_kernel<T, 8, kOnce, true, kT>), g, b, 0, st, a);
        else hipLaunchKernelGGL((combine_backward_kernel<T, 8, kOnce, false, kT>), g, b, 0, st, a);
        if (table && c.sums) hipLaunchKernelGGL(const_join_kernel<T>, join, dim3(kWide), 0, st, c);
    });
    return launched();
}

int moe_dispatch_backward(const void *grad_expand_x, const int32_t *assist_info, const int32_t *ep_recv_count,
                          const int32_t *expert_ids, const float *grad_expand_scales, const void *add,
                          const uint8_t *x_active_mask, int mask_kind, int ep_world, int bs, int experts_per_rank, int h,
                          int topk, int dtype, void *grad_x, float *grad_scales, void *stream)
{
    int rc = check_call(ep_world, bs, experts_per_rank, h, topk, dtype);
    if (rc) return rc;
    const long long N = (long long)ep_world * bs;
    if (!ep_recv_count || (N > 0 && (!grad_expand_x || !assist_info || !expert_ids || !grad_x))) return MOE_ERR_NULLPTR;
    if (N > 0 && !grad_expand_scales != !grad_scales) return MOE_ERR_NULLPTR;
    if ((rc = check_mask(x_active_mask, mask_kind, N))) return rc;
    if (!aligned(grad_expand_x, 2) || !aligned(assist_info, 4) || !aligned(ep_recv_count, 4) || !aligned(expert_ids, 4) ||
        !aligned(grad_expand_scales, 4) || !aligned(add, 2) || !aligned(grad_x, 2) || !aligned(grad_scales, 4))
        return MOE_ERR_ALIGN;
    if (N == 0) return MOE_OK;
    DispatchBackwardArgs a;
    a.r = routing_of(assist_info, ep_recv_count, expert_ids, x_active_mask, mask_kind, ep_world, bs, experts_per_rank, topk);
    a.grad = static_cast<const uint16_t *>(grad_expand_x);
    a.add = static_cast<const uint16_t *>(add);
    a.grad_scales_in = grad_expand_scales;
    a.out = static_cast<uint16_t *>(grad_x);
    a.grad_scales = grad_scales;
    a.h = h;
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const long long cols = threads_of(h) * kPiece;
    a.slices = N <= kFewTokens ? (int)std::min(16ll, (h + cols - 1) / cols) : 1;
    by_type(dtype, N * topk * h * 2, h, [&](auto type, auto once, auto threads) {
        constexpr int kT = decltype(threads)::value;
        hipLaunchKernelGGL((dispatch_backward_kernel<decltype(type), decltype(once)::value, kT>),
                           dim3((unsigned)(N * a.slices)), dim3(kT), 0, st, a);
    });
    return launched();
}

}  // extern "C"
