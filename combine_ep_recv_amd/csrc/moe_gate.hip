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
// A token's row stays in the registers of 16 or 64 lanes (see gate_kernel); the gradient takes a wavefront a token.

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
constexpr int kManyTokens = 32;            // tokens an expert, from which a token takes 16 lanes rather than 64
constexpr int kGateWaves = 8192;           // wavefronts of the gate: eight on each of 1024 SIMDs

struct GateArgs {
    const void *logits;
    const float *bias;
    const uint8_t *mask;
    int32_t *ids;
    float *weights;
    uint8_t *pair_mask;
    int tokens, experts, topk, groups, topk_groups, group_size, group_top2, renorm;
    uint32_t group_inv;                    // ceil(2^32 / group_size), 0 where that is 2^32: e / group_size for e < 2^11
    float scale;
};

__device__ __forceinline__ int group_of(uint32_t inv, int e) { return inv ? (int)__umulhi((uint32_t)e, inv) : e; }

// The two best values among the experts of each group, from v[E] in LDS, in the lanes that the group gets: `share`
// neighbouring ones, the largest power of two of which `groups` fit the token's lanes. All of them hold them on return.
template <class KEY, class PTR>
__device__ __forceinline__ void best_of_groups(PTR v, int groups, int size, int sub, int share, KEY &first, KEY &second)
{
    const KEY low = -(KEY)INFINITY;
    const int grp = sub / share;
    first = second = low;
    if (grp < groups) {
        for (int i = sub % share; i < size; i += share) {
            const KEY x = v[grp * size + i];
            second = max_of(second, x < first ? x : first);
            first = max_of(first, x);
        }
    }
    for (int d = 1; d < share; d *= 2) {
        const KEY f = __shfl_xor(first, d), s = __shfl_xor(second, d);
        second = max_of(max_of(second, s), f < first ? f : first);
        first = max_of(first, f);
    }
}

typedef __attribute__((address_space(3))) double lds_double;
typedef __attribute__((address_space(3))) const float lds_float;

template <class P>
__device__ __forceinline__ P uniform(P v)
{
    if constexpr (sizeof(P) == 8) {
        const uint64_t u = (uint64_t)v;
        return (P)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)u) |
                   (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(u >> 32)) << 32);
    } else {
        return (P)__builtin_amdgcn_readfirstlane((int)v);
    }
}

// exp(x - y) in binary64
__device__ __attribute__((noinline)) double exponential(float x, float y) { return exp((double)x - (double)y); }

// The choice for one token from binary64 scores, by a whole wavefront: lane k gets pair k's id. Rare but for equal sums
// (see gate_kernel), so it trades time for registers: the scores lie in LDS (v[experts], this wavefront's), the logits are
// read again (v holds them first). `bias` is LDS too, zeros where there is none. Not inlined: the constants of binary64's
// exponential would be kept in registers through gate_kernel's loop. Every argument is the same in all lanes.
template <class T, int SCORE>
__device__ __attribute__((noinline)) int choose_exactly(const typename T::raw *row_, lds_float *bias, int biased_, lds_double *v,
                                                        int experts_, int topk_, int groups_, int topk_groups_,
                                                        int group_size_, uint32_t group_inv_, int group_top2_)
{
    const typename T::raw *row = uniform(row_);
    const int biased = uniform(biased_), experts = uniform(experts_), topk = uniform(topk_), groups = uniform(groups_);
    const int topk_groups = uniform(topk_groups_), size = uniform(group_size_), top2 = uniform(group_top2_);
    const uint32_t inverse = uniform(group_inv_);
    const int lane = threadIdx.x % kWave;
    const double low = -(double)INFINITY;
    float top = -INFINITY;
    wave_fence();
#pragma unroll 4
    for (int e = lane; e < experts; e += kWave) {
        const float l = fmaxf(T::load(row[e]), -INFINITY);
        v[e] = l;
        top = fmaxf(top, l);
    }
    top = wave_max(top);
    double sum = 0;
    auto score = [&](float l) -> double {
        if (!(l > -INFINITY)) return 0.0;
        if (SCORE == MOE_SCORE_SOFTMAX) return exp(l == top ? 0.0 : (double)l - (double)top);
        return 1.0 / (1.0 + exp(-(double)l));
    };
    if (SCORE == MOE_SCORE_SOFTMAX) {
#pragma unroll 1
        for (int e = lane; e < experts; e += kWave) sum += score((float)v[e]);
        sum = wave_sum(sum);
    }
    const double inv = SCORE == MOE_SCORE_SOFTMAX && sum > 0 ? 1.0 / sum : 1.0;
    const bool by_score = biased || (groups > 1 && top2);    // what the groups are chosen by
#pragma unroll 1
    for (int e = lane; e < experts; e += kWave) {
        const float l = (float)v[e], b = bias[e];
        v[e] = !(l > -INFINITY && b > -INFINITY) ? low : (by_score ? score(l) * inv + (double)b : (double)l);
    }
    wave_fence();
    if (groups > 1) {
        int share = 1;
        while (share * 2 * groups <= kWave) share *= 2;
        double first, second;
        best_of_groups(v, groups, size, lane, share, first, second);
        double worth = top2 && second > low ? first + second : first;
        if (lane % share != 0) worth = low;
        unsigned long long kept = 0;
#pragma unroll 1
        for (int i = 0; i < topk_groups; ++i) {
            const double m = wave_max(worth);
            if (m == low) break;
            const int at = __ffsll((long long)__ballot(worth == m)) - 1;
            kept |= 1ull << (at / share);
            if (lane == at) worth = low;
        }
        wave_fence();
#pragma unroll 1
        for (int e = lane; e < experts; e += kWave) {
            if (!((kept >> group_of(inverse, e)) & 1)) v[e] = low;
            else if (!biased && v[e] > low) v[e] = T::load(row[e]);
        }
        wave_fence();
    }
    int id = -1;
    double best = low;
    uint32_t at = 0xffffffffu;
    auto scan = [&] {
        best = low;
        at = 0xffffffffu;
#pragma unroll 4
        for (int e = lane; e < experts; e += kWave) {
            const double x = v[e];
            at = x > best ? e : at;
            best = x > best ? x : best;
        }
    };
    scan();
#pragma unroll 1
    for (int k = 0; k < topk; ++k) {
        const double m = wave_max(best);
        if (m == low) break;
        const uint32_t e = wave_min(best == m ? at : 0xffffffffu);
        if (lane == k) id = (int)e;
        if (at == e) {
            v[e] = low;
            scan();
        }
    }
    return id;
}

// LANES lanes a token, 64 / LANES tokens a wavefront; lane `sub` of a token holds experts j * LANES + sub. Wavefronts
// stay for many tokens, with the bias in LDS and the next tokens' logits on their way.
//
// Choosing: each lane first sorts out the DEPTH best of its own PER experts (a maximum and medians of three for the
// values). A pick is then a maximum over the lanes' best, the lowest expert that has it, and one lane's list moving
// up; a lane whose list runs dry makes a new one from what it has below its last pick. 16 lanes a token make four
// tokens share each of these instructions; 64 make one token's way shorter, for calls with few tokens.
//
// Two experts' order may hang on the last bits of their scores, and has to come out as in binary64, whose
// exponentials cost about ten times fp32's. So the choice is made on fp32 scores, and made again on binary64 ones
// only where two neighbours in it, or the last one and the best left out, are closer than the fp32 scores may be off
// (u = 2^-24; the hardware's exp2 and reciprocal are off by 2 u). One such token costs 5.5 us, and the last one of a
// launch is waited for, so the bound is worth its care.
//   softmax  two exponentials, each off by 2.25 |x| u (a difference, a product, its constant) and 2 u, where
//            |x| e^x <= 0.37: 5.7 u of the largest score. The sum is the same for both: the difference of two scores
//            shares its error, E / 64 + 7 u for adding, 2 u and 2.25 |x| u, |x| averaged over the sum and so
//            at most 3.6 for 320 experts and 5.1 for 2048, and 2 u for its reciprocal. Below (E / 64 + 32) u together.
//   sigmoid  1.25 |x| s (1 - s) u <= 0.3 u, half of exp2's u (s (1 - s) <= 1/4), u of the sum and 2 u of the
//            reciprocal: below 4 u each.
// Either way half an ulp of each choice for its sum with the bias; for a group's sum of two, of each term and of the sum.
// Without a bias the logits themselves are compared, which needs neither.
// Of the tokens of a random bias one in two thousand is decided again. Equal sums always are: under a bias of zeros, or
// any constant one, every tie of logits among the picks. A third of 65536 tokens of 256 bf16 logits have one, and take 96
// us (fp16 logits 53), 37 and 35 with a random bias; 4096 tokens 14.5 and 11.0.
//
// What bounds it: vector instructions and their order, not memory. 65521 tokens of 304 experts (bf16, softmax, bias,
// 8 picks, a quarter of the tokens masked) take 47 us, 40 without the last binary64 look, for 30 MB of logits (6 us);
// the vector units are busy for 32 of them (1200 instructions for four tokens, with every list and pick). 4096 tokens
// of 256 experts in 8 groups take 11 to 14, 8.5 without that look; 8 tokens take 11, 3.5 of them on the card.
template <class T, int LANES, int PER, int WAVES, int SCORE>
__global__ __launch_bounds__(WAVES *kWave, LANES == 16 ? 4 : (PER <= 5 ? 5 : 1)) void gate_kernel(GateArgs a)
{
    constexpr int kTokens = kWave / LANES;                // tokens of a wavefront
    constexpr int DEPTH = PER < (LANES == 16 ? 4 : 2) ? PER : (LANES == 16 ? 4 : 2);
    // a wavefront's scratch: a row of doubles, or its tokens' rows of floats
    __shared__ double rows[WAVES][LANES * PER * (kTokens > 2 ? kTokens / 2 : 1)];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int sub = lane % LANES, stride = gridDim.x * WAVES * kTokens;
    const float low = -INFINITY, log2e = 1.44269504f;
    const typename T::raw *table = static_cast<const typename T::raw *>(a.logits);
    const bool by_score = a.bias || (a.groups > 1 && a.group_top2);
    __shared__ float bias[LANES * PER];
    for (int e = threadIdx.x; e < LANES * PER; e += WAVES * kWave) bias[e] = a.bias && e < a.experts ? a.bias[e] : 0.f;
    __syncthreads();
    typename T::raw next[PER];
    auto fetch = [&](int t) {                             // past a row or the last token: a value that is not used
        const typename T::raw *p = table + (size_t)min(t, a.tokens - 1) * a.experts + sub;
#pragma unroll
        for (int j = 0; j < PER; ++j) next[j] = p[min(j * LANES, a.experts - 1 - sub)];
    };
    auto active = [&](int t) -> bool { return t < a.tokens && (!a.mask || a.mask[t]); };
    int base = (blockIdx.x * WAVES + wave) * kTokens;     // the wavefront's first token
    bool on = active(base + lane / LANES), on_next = active(base + stride + lane / LANES);
    if (__ballot(on)) fetch(base + lane / LANES);
    for (; base < a.tokens; base += stride) {
        const int t = base + lane / LANES;
        const bool now = on;
        float l[PER], top = low;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            // a maximum with -infinity turns NaN into it
            l[j] = (now & (j * LANES + sub < a.experts)) ? fmaxf(T::load(next[j]), low) : low;
            top = fmaxf(top, l[j]);
        }
        on = on_next;
        if (__ballot(on)) fetch(t + stride);
        on_next = active(t + 2 * stride);
        top = wave_max<LANES>(top);
        float inv = 1.f, best = 1.f, c[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) c[j] = l[j];
        bool safe = true;
        if (SCORE == MOE_SCORE_SOFTMAX) {
            // Experts that are 64 apart add up first, then the four of those sums that are 16 apart, then 16 such: one
            // order, whatever the lanes, so that a token's weights do not change with the length of its batch.
            constexpr int kSums = kWave / LANES;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                c[j] = __builtin_amdgcn_exp2f((l[j] - top) * log2e);
                sum[j % kSums] += c[j];
            }
            const float four = LANES == 16 ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : sum_of_rows(sum[0]);
            inv = best = __builtin_amdgcn_rcpf(wave_sum<16>(four));
            safe = top < INFINITY;                        // logits of +infinity: NaN above
        } else if (by_score) {
#pragma unroll
            for (int j = 0; j < PER; ++j) c[j] = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(l[j] * -log2e));
        }
        const float room = (SCORE == MOE_SCORE_SIGMOID ? 8 : LANES * PER / kWave + 32) * 0x1p-24f * best + 0x1p-100f;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const float b = bias[j * LANES + sub], s = by_score ? __builtin_fmaf(c[j], inv, b) : l[j];
            c[j] = ((l[j] > low) & (b > low)) ? s : low;
        }
        if (a.groups > 1) {
            float *v = reinterpret_cast<float *>(rows[wave]) + lane / LANES * (LANES * PER);
            wave_fence();
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j * LANES + sub] = c[j];
            wave_fence();
            int share = 1;
            while (share * 2 * a.groups <= LANES) share *= 2;
            float first, second;
            best_of_groups(v, a.groups, a.group_size, sub, share, first, second);
            float worth = a.group_top2 && second > low ? first + second : first;
            // what the rounding of a sum's terms goes by: they may cancel, and those of any group bear on the order
            float size = 0.f;
            if (a.group_top2)
                size = wave_max<LANES>(second > low ? fabsf(first) + fabsf(second) : (first > low ? fabsf(first) : 0.f));
            if (!(size < INFINITY)) safe = false;         // a sum that fp32 does not hold, and binary64 does
            if (sub % share != 0) worth = low;
            unsigned long long kept = 0;
            int place = sub;
            asm volatile("" : "+v"(place));               // or the groups of all PER experts are kept in registers
            float above = INFINITY;
            for (int i = 0; i <= a.topk_groups; ++i) {
                const float m = wave_max<LANES>(worth);
                if (i == a.topk_groups) {
                    // whether the last kept group lies clear of the best one left out
                    size = fmaxf(size, fabsf(above));
                    if (by_score && m > low && !(above - m > 2.f * (room + 0x1.4p-23f * size))) safe = false;
                    break;
                }
                const uint32_t at = wave_min<LANES>(worth == m && m > low ? (uint32_t)sub : 64u);
                if (at < 64u) {
                    kept |= 1ull << (at / share);
                    above = m;
                }
                if (sub == (int)at) worth = low;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int grp = group_of(a.group_inv, j * LANES + place);
                const bool in = LANES == 16 ? (uint32_t)kept >> (grp & 31) & 1 : kept >> (grp & 63) & 1;
                const float x = a.bias ? c[j] : l[j];
                c[j] = in ? x : low;
            }
        }
        // the lane's list: values and their registers, best first
        float hv[DEPTH];
        uint32_t he[DEPTH];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            hv[i] = low;
            he[i] = 0;
        }
        auto insert = [&](float x, uint32_t e) {
#pragma unroll
            for (int i = DEPTH - 1; i > 0; --i) {
                he[i] = x > hv[i - 1] ? he[i - 1] : (x > hv[i] ? e : he[i]);
                hv[i] = __builtin_amdgcn_fmed3f(hv[i - 1], hv[i], x);
            }
            he[0] = x > hv[0] ? e : he[0];
            hv[0] = fmaxf(hv[0], x);
        };
#pragma unroll
        for (int j = 0; j < PER; ++j) insert(c[j], j);
        int id = -1, taken = 0;
        float mine = low, behind = low;                   // pick `sub`'s value, and the best one left out
        const int picks = a.topk + (a.bias ? 1 : 0);
        for (int k = 0; k < picks; ++k) {
            const float m = wave_max<LANES>(hv[0]);
            const uint32_t e = wave_min<LANES>(((hv[0] == m) & (m > low)) ? he[0] * LANES + sub : 0xffffffffu);
            if (k == a.topk) {
                behind = m;
                break;
            }
            if (sub == k) {
                id = (int)e;
                mine = m;
            }
            const bool won = (he[0] * LANES + sub == e) & (m > low);
            const float last = hv[0];
            const uint32_t lastj = he[0];
#pragma unroll
            for (int i = 0; i + 1 < DEPTH; ++i) {
                hv[i] = won ? hv[i + 1] : hv[i];
                he[i] = won ? he[i + 1] : he[i];
            }
            hv[DEPTH - 1] = won ? low : hv[DEPTH - 1];
            if constexpr (DEPTH < PER) {
                taken += won;
                const bool dry = won && taken % DEPTH == 0;
                if (__ballot(dry)) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        insert((dry & ((c[j] < last) | ((c[j] == last) & ((uint32_t)j > lastj)))) ? c[j] : low, j);
                    }
                }
            }
        }
        if (a.bias) {
            // (an infinity above another gives NaN, which is not above anything)
            const float right = __shfl_down(mine, 1), after = sub == a.topk - 1 ? behind : right;
            const bool clear_of = mine == low || mine - after > room + 0x1.4p-23f * fabsf(mine);
            if (sub < a.topk && !clear_of) safe = false;
        }
        unsigned long long redo = by_score ? __ballot(now && top > low && !safe) : 0;
        while (redo) {
            const int g = (__ffsll((long long)redo) - 1) / LANES;        // token g of the wavefront
            redo &= ~(((LANES == kWave ? 0ull : 1ull << (LANES % kWave)) - 1) << (g * LANES % kWave));
            const int mineid = choose_exactly<T, SCORE>(table + (size_t)(base + g) * a.experts, (lds_float *)bias,
                                                        a.bias != nullptr, (lds_double *)rows[wave], a.experts, a.topk, a.groups,
                                                        a.topk_groups, a.group_size, a.group_inv, a.group_top2);
            const int got = __shfl(mineid, sub);
            if (lane / LANES == g) id = got;
        }
        if (sub >= a.topk) id = -1;
        // lane k's score, from its logit
        float w = 0.f;
        const bool any = id >= 0;
        const float x = any ? fmaxf(T::load(table[(size_t)t * a.experts + id]), low) : 0.f;
        if (SCORE == MOE_SCORE_SOFTMAX) {
            if (__ballot(now && !(top < INFINITY))) {             // +infinities share it
                float many = 0.f;
#pragma unroll 1
                for (int e = sub; e < a.experts; e += LANES)
                    many += now && T::load(table[(size_t)t * a.experts + e]) == top ? 1.f : 0.f;
                many = wave_sum<LANES>(many);
                if (!(top < INFINITY)) inv = 1.f / many;
            }
            w = x == top ? 1.f : expf(x - top);
        } else {
            w = 1.f / (1.f + expf(-x));
        }
        if (!any) w = 0.f;
        const float total = a.renorm ? wave_sum<LANES>(w) : 0.f;
        w = a.renorm ? (total > 0.f ? w / total : 0.f) : w * inv;
        // scores below e^-80, whose sum fp32 may not hold: the weights of such a token in binary64
        const unsigned long long tiny = __ballot(any && (SCORE == MOE_SCORE_SOFTMAX ? x - top : x) < -80.f);
        if (tiny) {
            double d = SCORE == MOE_SCORE_SOFTMAX ? exponential(x == top ? 0.f : x, x == top ? 0.f : top)
                                                  : 1.0 / (1.0 + exponential(-x, 0.f));
            if (!any) d = 0.0;
            double all = d;
#pragma unroll
            for (int i = 1; i < LANES; i *= 2) all += __shfl_xor(all, i);
            const bool here = LANES == kWave || (tiny >> (lane / LANES * LANES) & 0xffff);
            if (here) w = (float)(a.renorm ? (all > 0.0 ? d / all : 0.0) : d * (double)inv);
        }
        w = any ? w * a.scale : 0.f;
        if (sub < a.topk && t < a.tokens) {
            const size_t at = (size_t)t * a.topk + sub;
            a.ids[at] = id;
            a.weights[at] = w;
            if (a.pair_mask) a.pair_mask[at] = any;
        }
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

// One wavefront per token. Lane k takes pair k; the pairs' gradients meet the experts in an LDS row, from which each lane
// writes its experts', VEC neighbouring ones at a time (two where rows of 16-bit logits start at 4 bytes: half as many
// loads and stores). The row of logits, where every expert needs its score, is on its way before anything else.
// Memory bounds long calls: 65521 tokens of 304 experts in bf16 with a gradient for every logit take 18 us, 4.2 TB/s of
// 76 MB; 4096 tokens of 256 experts in fp32 take 3.3 us on the card, and 9 with the call.
template <class T, int PER, int VEC, int WAVES, int SCORE, bool RENORM>
__global__ __launch_bounds__(WAVES *kWave) void gate_backward_kernel(GateGradArgs a)
{
    constexpr bool kDense = SCORE == MOE_SCORE_SOFTMAX && !RENORM;
    using raw = typename T::raw;
    typedef raw vec __attribute__((ext_vector_type(VEC)));
    typedef float fvec __attribute__((ext_vector_type(VEC)));
    __shared__ fvec rows[WAVES][PER * kWave];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int t = blockIdx.x * WAVES + wave;
    if (t >= a.tokens) return;
    const float low = -INFINITY, log2e = 1.44269504f;
    const raw *row = static_cast<const raw *>(a.logits) + (size_t)t * a.experts;
    const int groups = a.experts / VEC;                       // VEC divides experts
    vec in[PER];
    if (kDense) {
#pragma unroll
        for (int j = 0; j < PER; ++j) in[j] = reinterpret_cast<const vec *>(row)[min(j * kWave + lane, groups - 1)];
    }
    const size_t at = (size_t)t * a.topk + min(lane, a.topk - 1);
    int id = a.ids[at];
    float w = a.weights[at], g = a.grad[at];
    const bool mine = lane < a.topk && id >= 0 && id < a.experts;
    if (!mine) w = g = 0.f;
    const float dot = wave_sum(g * w);
    float d = RENORM ? w * (g - dot / a.scale) : a.scale * g;
    if (SCORE == MOE_SCORE_SIGMOID && mine) {
        const float l = T::load(row[id]);
        d *= 1.f / (1.f + expf(l));
        if (!RENORM) d *= 1.f / (1.f + expf(-l));
    }
    fvec *own = rows[wave];
#pragma unroll
    for (int j = 0; j < PER; ++j) own[j * kWave + lane] = fvec(0.f);
    wave_fence();
    if (mine) atomicAdd(reinterpret_cast<float *>(own) + id, d);          // ids of a token are distinct
    wave_fence();
    float s[PER][VEC], top = low, sum = 0.f, inv = 0.f;
    if (kDense) {
#pragma unroll
        for (int j = 0; j < PER; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                s[j][i] = j * kWave + lane < groups ? fmaxf(T::load(in[j][i]), low) : low;      // NaN too
                top = fmaxf(top, s[j][i]);
            }
        top = wave_max(top);
        const bool endless = !(top < INFINITY);               // logits of +infinity share the softmax
#pragma unroll
        for (int j = 0; j < PER; ++j)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float e = __builtin_amdgcn_exp2f((s[j][i] - top) * log2e);
                s[j][i] = endless ? (s[j][i] == top ? 1.f : 0.f) : (s[j][i] > low ? e : 0.f);
                sum += s[j][i];
            }
        sum = wave_sum(sum);
        inv = sum > 0.f && __ballot(mine) ? 1.f / sum : 0.f;  // a token without pairs gets nothing
    }
    raw *out = static_cast<raw *>(a.out) + (size_t)t * a.experts;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int e = j * kWave + lane;
        const fvec x = own[e];
        vec v;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float y = x[i];
            if (kDense) y = inv > 0.f ? s[j][i] * inv * (y - dot) : 0.f;
            v[i] = T::store(y);
        }
        if (e < groups) reinterpret_cast<vec *>(out)[e] = v;
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
    a.group_inv = (uint32_t)(((1ull << 32) + a.group_size - 1) / a.group_size);
    a.scale = scale;
    hipStream_t st = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    // 16 lanes a token where there are tokens enough to fill the card that way, and where they hold the row and the
    // picks. Measured, 64 against 16 lanes, sigmoid and bias: 256 experts 11.1 / 11.8 us at 4096 tokens, 14.9 / 12.2 at
    // 8192, 68 / 39 at 65536; 64 experts 6.8 / 6.7 us at 2048, 48 / 18 at 65536; 512 experts 90 / 87 at 65536.
    const bool four = tokens >= kManyTokens * experts && experts <= 320 && topk <= 16 && a.groups <= 16;
    by_type(dtype, [&](auto type) {
        using T = decltype(type);
        auto launch = [&](auto lanes, auto per, auto waves) {
            constexpr int L = decltype(lanes)::value, P = decltype(per)::value, V = decltype(waves)::value;
            constexpr int kEach = V * (kWave / L);                // tokens of a workgroup
            const dim3 g((unsigned)std::min((tokens + kEach - 1) / kEach, kGateWaves / V)), b(V * kWave);
            if (score == MOE_SCORE_SOFTMAX)
                hipLaunchKernelGGL((gate_kernel<T, L, P, V, MOE_SCORE_SOFTMAX>), g, b, 0, st, a);
            else
                hipLaunchKernelGGL((gate_kernel<T, L, P, V, MOE_SCORE_SIGMOID>), g, b, 0, st, a);
        };
        using std::integral_constant;
        using Few = integral_constant<int, 16>;
        using Four = integral_constant<int, 4>;
        if (!four) by_row(experts, [&](auto per, auto waves) { launch(integral_constant<int, kWave>(), per, waves); });
        else if (experts <= 64) launch(Few(), integral_constant<int, 4>(), Four());
        else if (experts <= 128) launch(Few(), integral_constant<int, 8>(), Four());
        else if (experts <= 256) launch(Few(), integral_constant<int, 16>(), Four());
        else launch(Few(), integral_constant<int, 20>(), Four());
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
    // pairs of 16-bit logits: rows of an even length from a 4-byte boundary
    const bool pairs = xs == 2 && experts % 2 == 0 && aligned(logits, 4) && aligned(grad_logits, 4);
    by_type(dtype, [&](auto type) {
        using T = decltype(type);
        auto launch = [&](auto per, auto vec, auto waves) {
            constexpr int P = decltype(per)::value, C = decltype(vec)::value, V = decltype(waves)::value;
            const dim3 g((unsigned)((tokens + V - 1) / V)), b(V * kWave);
            if (score == MOE_SCORE_SOFTMAX && renormalize)
                hipLaunchKernelGGL((gate_backward_kernel<T, P, C, V, MOE_SCORE_SOFTMAX, true>), g, b, 0, st, a);
            else if (score == MOE_SCORE_SOFTMAX)
                hipLaunchKernelGGL((gate_backward_kernel<T, P, C, V, MOE_SCORE_SOFTMAX, false>), g, b, 0, st, a);
            else if (renormalize)
                hipLaunchKernelGGL((gate_backward_kernel<T, P, C, V, MOE_SCORE_SIGMOID, true>), g, b, 0, st, a);
            else
                hipLaunchKernelGGL((gate_backward_kernel<T, P, C, V, MOE_SCORE_SIGMOID, false>), g, b, 0, st, a);
        };
        using std::integral_constant;
        using One = integral_constant<int, 1>;
        using Two = integral_constant<int, 2>;
        using Four = integral_constant<int, 4>;
        if constexpr (sizeof(typename T::raw) == 2) {
            if (pairs) {
                if (experts <= 128) launch(One(), Two(), Four());
                else if (experts <= 256) launch(Two(), Two(), Four());
                else if (experts <= 384) launch(integral_constant<int, 3>(), Two(), Four());
                else if (experts <= 512) launch(Four(), Two(), Four());
                else if (experts <= 1024) launch(integral_constant<int, 8>(), Two(), Four());
                else launch(integral_constant<int, 16>(), Two(), One());
                return;
            }
        }
        by_row(experts, [&](auto per, auto waves) { launch(per, One(), waves); });
    });
    return launched();
}

}  // extern "C"
