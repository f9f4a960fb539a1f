// moe_gate.hip -- the gate in front of dispatch, forward and backward (gfx950, wave64).
//
// Forward, for a token's logits l over E experts:
//   s = softmax(l) or sigmoid(l), logits of -infinity and NaN left out;  c = s + bias (order of l without a bias);
//   the best groups by their experts' c, then the K largest c of those groups, ties to the lower id;
//   w_k = scale * s_k, divided by the sum of the K chosen s where renormalised.
// Backward, with g = dL/dw, D = sum_k g_k w_k:
//   softmax, renormalised   dl_k = w_k (g_k - D / scale), every other logit 0
//   sigmoid, renormalised   dl_k = w_k (g_k - D / scale) (1 - s_k)
//   sigmoid                 dl_k = scale g_k s_k (1 - s_k)
//   softmax                 dl_e = s_e (scale g_e - D), g_e = 0 where e was not chosen
//
// One wavefront per token, the row in registers (expert j * 64 + lane in register j of a lane), so that a token
// needs no barrier and a single-token call no second pass.

#include "moe_types.h"

#include <limits.h>

#include <algorithm>
#include <cmath>

namespace {

using namespace moe_detail;

constexpr int kMaxGateExperts = 2048;      // 1024 real ones and as many special ids
constexpr int kMaxGateTopk = 64;           // lane k of a wavefront holds pair k
constexpr int kMaxGroups = 64;             // one bit each in the mask of kept groups
constexpr long long kMaxTokens = (1ll << 24) - 1;   // dispatch's limit

struct GateArgs {
    const void *logits;
    const float *bias;
    const uint8_t *mask;
    int32_t *ids;
    float *weights;
    uint8_t *pair_mask;
    int tokens, experts, topk, groups, topk_groups, group_size, group_top2, renorm;
    uint64_t group_inv;                    // ceil(2^32 / group_size): e / group_size for e < 2^11
    float scale;
};

// The K largest of c[PER] per lane over the wavefront, in descending order, ties to the lower id (register j of
// lane l holds expert j * 64 + l). Lane k gets pair k's id, -1 where nothing above -infinity is left.
template <int PER, class KEY>
__device__ __forceinline__ int pick(KEY (&c)[PER], int K, int lane)
{
    const KEY low = -(KEY)INFINITY;
    int id = -1;
    for (int k = 0; k < K; ++k) {
        KEY m = c[0];
#pragma unroll
        for (int j = 1; j < PER; ++j) m = max_of(m, c[j]);
        m = wave_max(m);
        if (m == low) break;
        int e = -1;
#pragma unroll
        for (int j = PER - 1; j >= 0; --j) {
            const unsigned long long b = __ballot(c[j] == m);
            if (b) e = j * kWave + __ffsll((long long)b) - 1;
        }
        if (lane == k) id = e;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (e == j * kWave + lane) c[j] = low;
    }
    return id;
}

// The kept groups as a bit mask. v: each expert's value (unavailable: -infinity), copied through `row` in LDS so
// that a group's experts, wherever their lanes are, are read by the lanes that the group gets.
template <int PER, class KEY>
__device__ __forceinline__ unsigned long long keep_groups(const KEY (&v)[PER], KEY *row, const GateArgs &a, int lane)
{
    const KEY low = -(KEY)INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) row[j * kWave + lane] = v[j];
    wave_fence();
    int share = 1;                                  // lanes of a group: the largest power of two that fits
    while (share * 2 * a.groups <= kWave) share *= 2;
    const int grp = lane / share, sub = lane % share;
    KEY first = low, second = low;
    if (grp < a.groups) {
        for (int i = sub; i < a.group_size; i += share) {
            const KEY x = row[grp * a.group_size + i];
            second = max_of(second, x < first ? x : first);
            first = max_of(first, x);
        }
    }
    for (int d = 1; d < share; d *= 2) {
        const KEY f = __shfl_xor(first, d), s = __shfl_xor(second, d);
        second = max_of(max_of(second, s), f < first ? f : first);
        first = max_of(first, f);
    }
    KEY score = a.group_top2 && second > low ? first + second : first;
    if (sub != 0 || grp >= a.groups) score = low;
    unsigned long long kept = 0;
    for (int i = 0; i < a.topk_groups; ++i) {
        const KEY m = wave_max(score);
        if (m == low) break;
        const int at = __ffsll((long long)__ballot(score == m)) - 1;
        kept |= 1ull << (at / share);
        if (lane == at) score = low;
    }
    wave_fence();
    return kept;
}

template <class T, int PER, int WAVES, int SCORE>
__global__ __launch_bounds__(WAVES *kWave) void gate_kernel(GateArgs a)
{
    __shared__ double rows[WAVES][PER * kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int t = blockIdx.x * WAVES + wave;
    if (t >= a.tokens) return;
    const float low = -INFINITY;
    int id = -1;
    float w = 0.f;
    if (!a.mask || a.mask[t]) {
        const typename T::raw *row = static_cast<const typename T::raw *>(a.logits) + (size_t)t * a.experts;
        float l[PER], b[PER];
        float top = low;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * kWave + lane;
            l[j] = e < a.experts ? T::load(row[e]) : low;
            b[j] = a.bias && e < a.experts ? a.bias[e] : 0.f;
            if (!(l[j] > low)) l[j] = low;                      // NaN too
            top = fmaxf(top, l[j]);
        }
        top = wave_max(top);
        double s[PER], sum = 0, c[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (SCORE == MOE_SCORE_SOFTMAX) {
                s[j] = l[j] > low ? exp(l[j] == top ? 0.0 : (double)l[j] - (double)top) : 0.0;
                sum += s[j];
            } else {
                s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
            }
        }
        sum = SCORE == MOE_SCORE_SOFTMAX ? wave_sum(sum) : 1.0;
        const double inv = sum > 0 ? 1.0 / sum : 0.0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            if (SCORE == MOE_SCORE_SOFTMAX) s[j] *= inv;
            c[j] = l[j] > low && b[j] > low ? (a.bias ? s[j] + (double)b[j] : (double)l[j]) : (double)low;
        }
        if (a.groups > 1) {
            double v[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j)
                v[j] = c[j] > (double)low && !a.bias && a.group_top2 ? s[j] : c[j];
            const unsigned long long kept = keep_groups<PER>(v, rows[wave], a, lane);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int grp = (int)((j * kWave + lane) * a.group_inv >> 32);
                if (!((kept >> (grp & 63)) & 1)) c[j] = (double)low;
            }
        }
        id = pick<PER>(c, a.topk, lane);
        double mine = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const double x = __shfl(s[j], id & 63);
            if (id >> 6 == j) mine = x;
        }
        if (id < 0) mine = 0;
        if (a.renorm) {
            const double total = wave_sum(mine);
            mine = total > 0 ? mine / total : 0.0;
        }
        w = (float)(mine * (double)a.scale);
    }
    if (lane < a.topk) {
        const size_t at = (size_t)t * a.topk + lane;
        a.ids[at] = id;
        a.weights[at] = w;
        if (a.pair_mask) a.pair_mask[at] = id >= 0;
    }
}

struct GateGradArgs {
    const void *logits;
    const int32_t *ids;
    const float *weights, *grad;
    void *out;
    int tokens, experts, topk;
    float scale;
};

template <class T, int PER, int WAVES, int SCORE, bool RENORM>
__global__ __launch_bounds__(WAVES *kWave) void gate_backward_kernel(GateGradArgs a)
{
    __shared__ float rows[WAVES][PER * kWave];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int t = blockIdx.x * WAVES + wave;
    if (t >= a.tokens) return;
    const float low = -INFINITY;
    const typename T::raw *row = static_cast<const typename T::raw *>(a.logits) + (size_t)t * a.experts;
    int id = -1;
    float w = 0.f, g = 0.f;
    if (lane < a.topk) {
        const size_t at = (size_t)t * a.topk + lane;
        id = a.ids[at];
        if (id < 0 || id >= a.experts) id = -1;
        else {
            w = a.weights[at];
            g = a.grad[at];
        }
    }
    const float dot = wave_sum(g * w);
    float d = RENORM ? w * (g - dot / a.scale) : a.scale * g;
    if (SCORE == MOE_SCORE_SIGMOID && id >= 0) {
        const float l = T::load(row[id]);
        d *= 1.f / (1.f + expf(l));
        if (!RENORM) d *= 1.f / (1.f + expf(-l));
    }
    float *mine = rows[wave];
#pragma unroll
    for (int j = 0; j < PER; ++j) mine[j * kWave + lane] = 0.f;
    wave_fence();
    if (id >= 0) atomicAdd(&mine[id], d);          // ids of a token are distinct
    wave_fence();
    typename T::raw *out = static_cast<typename T::raw *>(a.out) + (size_t)t * a.experts;
    if (SCORE == MOE_SCORE_SOFTMAX && !RENORM) {
        const bool any = __ballot(id >= 0) != 0;
        float l[PER], top = low, sum = 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * kWave + lane;
            l[j] = any && e < a.experts ? T::load(row[e]) : low;
            if (!(l[j] > low)) l[j] = low;
            top = fmaxf(top, l[j]);
        }
        top = wave_max(top);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            l[j] = l[j] > low ? expf(l[j] == top ? 0.f : l[j] - top) : 0.f;
            sum += l[j];
        }
        sum = wave_sum(sum);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * kWave + lane;
            if (e < a.experts) out[e] = T::store(l[j] * inv * (mine[e] - dot));
        }
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = j * kWave + lane;
            if (e < a.experts) out[e] = T::store(mine[e]);
        }
    }
}

int check_gate(int tokens, int experts, int topk, int dtype, int score, float scale)
{
    if (tokens < 0 || tokens > kMaxTokens || experts < 1 || experts > kMaxGateExperts || topk < 1 ||
        topk > kMaxGateTopk || topk > experts)
        return MOE_ERR_SHAPE;
    if (dtype != MOE_FP16 && dtype != MOE_BF16 && dtype != MOE_FP32) return MOE_ERR_DTYPE;
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) return MOE_ERR_SHAPE;
    if (!std::isfinite(scale) || scale == 0.f) return MOE_ERR_SHAPE;
    return MOE_OK;
}

// Registers per lane for a row of `experts`, and wavefronts per workgroup (one where the row's LDS copy is large).
template <class F>
void by_row(int experts, F f)
{
    const int per = (experts + kWave - 1) / kWave;
    using std::integral_constant;
    if (per <= 1) f(integral_constant<int, 1>(), integral_constant<int, 4>());
    else if (per <= 2) f(integral_constant<int, 2>(), integral_constant<int, 4>());
    else if (per <= 4) f(integral_constant<int, 4>(), integral_constant<int, 4>());
    else if (per <= 5) f(integral_constant<int, 5>(), integral_constant<int, 4>());
    else if (per <= 8) f(integral_constant<int, 8>(), integral_constant<int, 4>());
    else if (per <= 16) f(integral_constant<int, 16>(), integral_constant<int, 1>());
    else f(integral_constant<int, 32>(), integral_constant<int, 1>());
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

int moe_gate(const void *logits, const float *bias, const uint8_t *token_mask, int tokens, int experts, int topk,
             int dtype, int score, int groups, int topk_groups, int group_score, int renormalize, float scale,
             int32_t *expert_ids, float *expert_scales, uint8_t *pair_mask, void *stream)
{
    const int rc = check_gate(tokens, experts, topk, dtype, score, scale);
    if (rc) return rc;
    if (groups < 1 || groups > kMaxGroups || experts % groups || topk_groups < 1 || topk_groups > groups ||
        topk > topk_groups * (experts / groups))
        return MOE_ERR_SHAPE;
    if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2) return MOE_ERR_SHAPE;
    if (tokens == 0) return MOE_OK;
    if (!logits || !expert_ids || !expert_scales) return MOE_ERR_NULLPTR;
    if (!aligned(logits, dtype == MOE_FP32 ? 4 : 2) || !aligned(bias, 4) || !aligned(expert_ids, 4) ||
        !aligned(expert_scales, 4))
        return MOE_ERR_ALIGN;
    GateArgs a;
    a.logits = logits;
    a.bias = bias;
    a.mask = token_mask;
    a.ids = expert_ids;
    a.weights = expert_scales;
    a.pair_mask = pair_mask;
    a.tokens = tokens;
    a.experts = experts;
    a.topk = topk;
    a.groups = topk_groups < groups ? groups : 1;   // every group kept: no grouping
    a.topk_groups = topk_groups;
    a.group_size = experts / groups;
    a.group_top2 = group_score == MOE_GROUP_TOP2;
    a.renorm = renormalize != 0;
    a.group_inv = ((1ull << 32) + a.group_size - 1) / a.group_size;
    a.scale = scale;
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) {
        by_row(experts, [&](auto per, auto waves) {
            using T = decltype(type);
            constexpr int P = decltype(per)::value, V = decltype(waves)::value;
            const dim3 g((unsigned)((tokens + V - 1) / V)), b(V * kWave);
            if (score == MOE_SCORE_SOFTMAX)
                hipLaunchKernelGGL((gate_kernel<T, P, V, MOE_SCORE_SOFTMAX>), g, b, 0, st, a);
            else
                hipLaunchKernelGGL((gate_kernel<T, P, V, MOE_SCORE_SIGMOID>), g, b, 0, st, a);
        });
    });
    return launched();
}

int moe_gate_backward(const void *logits, const int32_t *expert_ids, const float *expert_scales,
                      const float *grad_scales, int tokens, int experts, int topk, int dtype, int score,
                      int renormalize, float scale, void *grad_logits, void *stream)
{
    const int rc = check_gate(tokens, experts, topk, dtype, score, scale);
    if (rc) return rc;
    if (tokens == 0) return MOE_OK;
    if (!logits || !expert_ids || !expert_scales || !grad_scales || !grad_logits) return MOE_ERR_NULLPTR;
    const size_t xs = dtype == MOE_FP32 ? 4 : 2;
    if (!aligned(logits, xs) || !aligned(expert_ids, 4) || !aligned(expert_scales, 4) || !aligned(grad_scales, 4) ||
        !aligned(grad_logits, xs))
        return MOE_ERR_ALIGN;
    GateGradArgs a;
    a.logits = logits;
    a.ids = expert_ids;
    a.weights = expert_scales;
    a.grad = grad_scales;
    a.out = grad_logits;
    a.tokens = tokens;
    a.experts = experts;
    a.topk = topk;
    a.scale = scale;
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_type(dtype, [&](auto type) {
        by_row(experts, [&](auto per, auto waves) {
            using T = decltype(type);
            constexpr int P = decltype(per)::value, V = decltype(waves)::value;
            const dim3 g((unsigned)((tokens + V - 1) / V)), b(V * kWave);
            if (score == MOE_SCORE_SOFTMAX && renormalize)
                hipLaunchKernelGGL((gate_backward_kernel<T, P, V, MOE_SCORE_SOFTMAX, true>), g, b, 0, st, a);
            else if (score == MOE_SCORE_SOFTMAX)
                hipLaunchKernelGGL((gate_backward_kernel<T, P, V, MOE_SCORE_SOFTMAX, false>), g, b, 0, st, a);
            else if (renormalize)
                hipLaunchKernelGGL((gate_backward_kernel<T, P, V, MOE_SCORE_SIGMOID, true>), g, b, 0, st, a);
            else
                hipLaunchKernelGGL((gate_backward_kernel<T, P, V, MOE_SCORE_SIGMOID, false>), g, b, 0, st, a);
        });
    });
    return launched();
}

}  // extern "C"
