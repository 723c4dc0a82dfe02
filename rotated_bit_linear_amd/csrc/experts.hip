// The operators around the experts' products: the router that chooses each token's experts, the plan that
// sorts the choices by expert, and the weighted sum that brings the experts' rows back to the tokens.
#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

#include "elem_load.hpp"
#include "experts.hpp"
#include "kernels.hpp"

namespace convrot {
namespace {

// ------------------------------------------------------------------------------ router ----

// largest of a wave's 32-bit values, in every lane
__device__ __forceinline__ uint32_t wave_max(uint32_t x)
{
    auto step = [&](uint32_t y) { x = x > y ? x : y; };
    step(__builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true));
    step(__builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true));
    step(__builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true));
    step(__builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true));
    step(__builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));
    step(__builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));
    return __builtin_amdgcn_readlane(x, 63);
}

// a double's bits in an order of unsigned numbers; 0 is below every number's (and no number's own)
__device__ __forceinline__ uint64_t ordered(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);      // -0 equals 0
    return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}

template <int CTRL>
__device__ __forceinline__ double dpp(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}
// the value of the other half of 2^(lg + 1) lanes, where each half of 2^lg holds one value: by quads, half
// rows and rows of 16 lanes, above by a shuffle
__device__ __forceinline__ double other_half(double v, int lg)
{
    switch (lg) {
    case 0: return dpp<0xB1>(v);                      // quad_perm 1 0 3 2
    case 1: return dpp<0x4E>(v);                      // quad_perm 2 3 0 1
    case 2: return dpp<0x141>(v);                     // row_half_mirror
    case 3: return dpp<0x140>(v);                     // row_mirror
    default: return __shfl_xor(v, 1 << lg);
    }
}
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int lg = 0; lg < 6; lg++) v += other_half(v, lg);
    return v;
}
__device__ __forceinline__ double read_lane(double v, int lane)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}
// 1 / (1 + exp(-x)) in FP64: the instruction's estimate of the reciprocal and two Newton steps, within 2^-51.
// The denominator is held times 2^-60, so that it, its reciprocal and their products are normal numbers up to the
// exponential's overflow (x of -709.78; 0 from there on); the factor is exact, but for scores below the normal range.
__device__ __forceinline__ double sigmoid_f64(float x)
{
    const double d = fma(exp(-(double)x), 0x1p-60, 0x1p-60);
    double y = __builtin_amdgcn_rcp(d);
    y = fma(fma(-d, y, 1.0), y, y);
    y = fma(fma(-d, y, 1.0), y, y);
    return d < INFINITY ? y * 0x1p-60 : 0.0;
}

// One wave a token; lane l holds experts l, l + 64, ...
// Which experts are chosen has to follow from the scores in FP64: it must not turn on a rounding.  Without a
// bias the logits order the experts as the scores do, and are compared themselves.  Otherwise keys (and
// groups' values) are computed in FP32 first, off by less than kSure / 4 of max(1, |key|); where every two
// keys whose order matters are further apart than kSure, that order is FP64's, and FP64 computes the chosen
// experts' scores alone, a lane each.  Where they are not, the token is done again in FP64.  (kSure 2^-17;
// sigmoid: an exponent's argument off by 2^-24 of it, exponential, addition and reciprocal by 2^-23 each;
// softmax: a sum of up to 512 powers in 14 levels, 2^-20; the bias' addition 2^-24.)
// The choice: each lane sorts its own keys, then k times the wave's largest head, the lowest expert where
// several have it, is taken.  Bound by its instructions: 19989 tokens, 256 experts in 8 groups, sigmoid with a
// bias, 8 choices 28 us in a captured loop (the first form, wholly in FP64, 42); 64 experts, softmax 12.
constexpr int kRouteWaves = 4;
constexpr float kSure = 0x1p-17f;

__device__ __forceinline__ uint32_t ordered32(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);                     // -0 equals 0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered32(uint32_t o)
{
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ float read_lane(float v, int lane)
{
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
__device__ __forceinline__ float other_half(float v, int lg)
{
    const int x = (int)__float_as_uint(v);
    switch (lg) {
    case 0: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0xB1, 0xF, 0xF, true));
    case 1: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0x4E, 0xF, 0xF, true));
    case 2: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0x141, 0xF, 0xF, true));
    case 3: return __uint_as_float(__builtin_amdgcn_update_dpp(0, x, 0x140, 0xF, 0xF, true));
    default: return __shfl_xor(v, 1 << lg);
    }
}

// Groups whose experts may be chosen, bit g << lanes_lg for group g, from the experts' values in LDS (-inf
// where there is none).  sure is cleared where `margin` leaves it open.
template <bool FUZZY, class F>
__device__ __forceinline__ uint64_t best_groups(const RouteLaunch &a, const F *values, F margin, int lane, bool &sure)
{
    const int size = a.group_size, per = 1 << a.lanes_lg, g = lane >> a.lanes_lg;
    F b1 = -INFINITY, b2 = -INFINITY;
    auto second = [](F x, F y) { return x < y ? x : y; };
    auto first = [](F x, F y) { return x > y ? x : y; };
    if (g < a.G)
        for (int x = lane & (per - 1); x < size; x += per) {
            const F v = values[g * size + x];
            b2 = first(b2, second(b1, v));
            b1 = first(b1, v);
        }
    for (int lg = 0; lg < a.lanes_lg; lg++) {
        const F o1 = other_half(b1, lg), o2 = other_half(b2, lg);
        b2 = first(first(b2, o2), second(b1, o1));
        b1 = first(b1, o1);
    }
    const bool two = a.group_sum == 2 && b2 > -INFINITY;
    const F v = two ? b1 + b2 : b1;
    auto size_of = [&](F x) { return x < 0 ? -x : x; };
    const F slack = margin * first(F(1), size_of(v));
    int better = 0, perhaps = 0;                      // groups that come before this one, that may
    for (int o = 0; o < a.G; o++) {
        const F w = read_lane(v, o << a.lanes_lg);
        if constexpr (FUZZY) {
            better += w > v + slack;
            perhaps += o != g && w > v - slack;
        } else {
            better += w > v || (w == v && o < g);
        }
    }
    if constexpr (FUZZY) {
        // a sum that cancels, or overflows FP32, is not as near as the margin says
        const F part = two ? first(size_of(b1), size_of(b2)) : size_of(b1);
        const bool far = !(part <= 2 * first(F(1), size_of(v))) || v == INFINITY;
        sure = sure && __builtin_amdgcn_ballot_w64(
                           g < a.G && (far || (perhaps >= a.top_groups && better < a.top_groups))) == 0;
    }
    return __builtin_amdgcn_ballot_w64(g < a.G && better < a.top_groups);
}

template <int DT, int NE>
__global__ __launch_bounds__(64 * kRouteWaves)
void route_kernel(const RouteLaunch a)
{
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;
    const auto *row = static_cast<const typename Elem<DT>::T *>(a.logits) + t * a.ld;
    auto wave_fence = [] {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };

    // e / group_size for e < 512: the factor is off by less than 2^-20 of one
    auto group_of = [&](int e) { return e < a.E ? (int)((uint32_t)e * a.group_factor >> 20) : 0; };

    float l[NE], b[NE];
    uint32_t key[NE], top = 0;
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = 64 * i + lane;
        l[i] = e < a.E ? Elem<DT>::cvt(row[e]) : -INFINITY;
        b[i] = a.bias && e < a.E ? a.bias[e] : 0.0f;
    }
    const bool grouped = a.top_groups < a.G;
    const bool all_scores = a.bias || (grouped && a.group_sum == 2);
    float most = 0.0f;
    if (!a.sigmoid) {
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const uint32_t o = l[i] > -INFINITY ? ordered32(l[i]) : 0u;
            top = top > o ? top : o;
        }
        most = unordered32(wave_max(top));
    }
    // a logit of -inf or NaN, and a key of either, is never chosen
    auto valid = [&](int i, auto v) { return l[i] > -INFINITY && v > -INFINITY; };
    // exp(l - most), 1 where they are equal (infinite or not)
    auto power = [&](float x) { return x == most ? 1.0 : exp((double)x - (double)most); };

    bool sure = true;
    float value[NE];
    if (all_scores) {
        constexpr float log2e = 0x1.715476p+0f;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < NE; i++)
                value[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-l[i] * log2e));
        } else {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NE; i++) {
                value[i] = l[i] == most ? 1.0f : l[i] > -INFINITY ? __builtin_amdgcn_exp2f((l[i] - most) * log2e) : 0.0f;
                sum += value[i];
            }
#pragma unroll
            for (int lg = 0; lg < 6; lg++) sum += other_half(sum, lg);
            sum = __builtin_amdgcn_rcpf(sum);
#pragma unroll
            for (int i = 0; i < NE; i++) value[i] *= sum;
        }
#pragma unroll
        for (int i = 0; i < NE; i++) value[i] += b[i];
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const float v = a.bias ? value[i] : l[i];
        key[i] = valid(i, v) ? ordered32(v) : 0u;
    }
    if (grouped) {
        float *values = reinterpret_cast<float *>(lds + wave * a.E);
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int e = 64 * i + lane;
            const float v = all_scores ? value[i] : l[i];
            if (e < a.E) values[e] = valid(i, v) ? v : -INFINITY;
        }
        wave_fence();
        const uint64_t kept = all_scores ? best_groups<true>(a, values, kSure, lane, sure)
                                         : best_groups<false>(a, values, 0.0f, lane, sure);
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int e = 64 * i + lane;
            if (!(kept >> (group_of(e) << a.lanes_lg) & 1)) key[i] = 0;
        }
    }

    int id = -1;                                      // lane j: choice j
    if (sure) {
        // each lane's keys from the largest down, with the places that they come from
        int at[NE];
#pragma unroll
        for (int i = 0; i < NE; i++) at[i] = i;
        auto exchange = [&](int x, int y) {
            const bool swap = key[x] < key[y] || (key[x] == key[y] && at[x] > at[y]);
            const uint32_t k0 = key[x], k1 = key[y];
            const int a0 = at[x], a1 = at[y];
            key[x] = swap ? k1 : k0; key[y] = swap ? k0 : k1;
            at[x] = swap ? a1 : a0; at[y] = swap ? a0 : a1;
        };
        if constexpr (NE == 2) exchange(0, 1);
        if constexpr (NE >= 4) {
#pragma unroll
            for (int o = 0; o < NE; o += 4) {
                exchange(o, o + 1); exchange(o + 2, o + 3); exchange(o, o + 2); exchange(o + 1, o + 3); exchange(o + 1, o + 2);
            }
        }
        if constexpr (NE == 8) {
#pragma unroll
            for (int i = 0; i < 4; i++) exchange(i, i + 4);
            exchange(2, 4); exchange(3, 5);
            exchange(1, 2); exchange(3, 4); exchange(5, 6);
        }
        float last = INFINITY;
        for (int j = 0; j <= a.k; j++) {              // one more than is chosen: is the border clear
            const uint32_t best = wave_max(key[0]);
            if (best == 0) break;                     // none left
            if (a.bias) {
                const float v = unordered32(best);
                sure = sure && last - v > kSure * fmaxf(1.0f, fabsf(v));
                last = v;
            }
            if (j == a.k) break;
            uint64_t have = __builtin_amdgcn_ballot_w64(key[0] == best);
            int from = __builtin_ctzll(have);
            int e = 64 * __builtin_amdgcn_readlane(at[0], from) + from;
            if (have & (have - 1)) {                  // several lanes: the lowest expert
                e = (int)~wave_max(key[0] == best ? ~(uint32_t)(64 * at[0] + lane) : 0u);
                from = e & 63;
            }
            id = lane == j ? e : id;
            const bool mine = lane == from;
#pragma unroll
            for (int i = 0; i + 1 < NE; i++) {
                key[i] = mine ? key[i + 1] : key[i];
                at[i] = mine ? at[i + 1] : at[i];
            }
            key[NE - 1] = mine ? 0u : key[NE - 1];
        }
        sure = __builtin_amdgcn_readfirstlane(sure);
    }
    double norm = 1.0;                                // softmax: 1 / sum of the powers
    if (!a.sigmoid && (!a.renorm || !sure)) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NE; i++) sum += l[i] > -INFINITY ? power(l[i]) : 0.0;
        norm = 1.0 / wave_sum(sum);
    }
    if (!sure) {
        uint32_t hi[NE], lo[NE];
        double exact[NE];
#pragma unroll
        for (int i = 0; i < NE; i++) {
            exact[i] = (a.sigmoid ? sigmoid_f64(l[i]) : power(l[i]) * norm) + (double)b[i];
            const double v = a.bias ? exact[i] : (double)l[i];
            const uint64_t k = ordered(v);
            hi[i] = valid(i, v) ? (uint32_t)(k >> 32) : 0u;           // a number's upper half is not 0
            lo[i] = (uint32_t)k;
        }
        if (grouped) {
            double *values = lds + wave * a.E;
            wave_fence();
#pragma unroll
            for (int i = 0; i < NE; i++) {
                const int e = 64 * i + lane;
                if (e < a.E) values[e] = hi[i] ? exact[i] : -INFINITY;
            }
            wave_fence();
            const uint64_t kept = best_groups<false>(a, values, 0.0, lane, sure);
#pragma unroll
            for (int i = 0; i < NE; i++) {
                const int e = 64 * i + lane;
                if (!(kept >> (group_of(e) << a.lanes_lg) & 1)) hi[i] = 0;
            }
        }
        id = -1;
        for (int j = 0; j < a.k; j++) {
            uint32_t best = 0, low = 0, inv = 0;
#pragma unroll
            for (int i = 0; i < NE; i++) best = best > hi[i] ? best : hi[i];
            best = wave_max(best);
            if (best == 0) break;
#pragma unroll
            for (int i = 0; i < NE; i++) low = hi[i] == best && lo[i] > low ? lo[i] : low;
            low = wave_max(low);
#pragma unroll
            for (int i = 0; i < NE; i++) {
                const uint32_t x = ~(uint32_t)(64 * i + lane);
                inv = hi[i] == best && lo[i] == low && x > inv ? x : inv;
            }
            const int e = (int)~wave_max(inv);
#pragma unroll
            for (int i = 0; i < NE; i++) hi[i] = 64 * i + lane == e ? 0u : hi[i];
            id = lane == j ? e : id;
        }
    }
    // the chosen experts' own scores, a lane each
    const float chosen = id < 0 ? 0.0f : Elem<DT>::cvt(row[id]);
    const double s = id < 0 ? 0.0 : a.sigmoid ? sigmoid_f64(chosen) : power(chosen) * norm;
    double w = s * (double)a.scale;
    if (a.renorm) {
        const double sum = wave_sum(s);
        w = sum > 0.0 ? w / sum : 0.0;
    }
    if (lane < a.k) {
        a.ids[t * a.k + lane] = id;
        a.weights[t * a.k + lane] = (float)w;
    }
}

template <int DT>
hipError_t launch_route_of(const RouteLaunch &a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.T + kRouteWaves - 1) / kRouteWaves)), threads(64 * kRouteWaves);
    const size_t lds = a.top_groups < a.G ? (size_t)kRouteWaves * a.E * sizeof(double) : 0;
    if (a.E <= 64) hipLaunchKernelGGL((route_kernel<DT, 1>), grid, threads, lds, st, a);
    else if (a.E <= 128) hipLaunchKernelGGL((route_kernel<DT, 2>), grid, threads, lds, st, a);
    else if (a.E <= 256) hipLaunchKernelGGL((route_kernel<DT, 4>), grid, threads, lds, st, a);
    else hipLaunchKernelGGL((route_kernel<DT, 8>), grid, threads, lds, st, a);
    return hipGetLastError();
}

// -------------------------------------------------------------------------------- plan ----

// A stable counting sort.  A workgroup takes a run of slots, each of its waves a part of the run in
// order.  Slots of no expert here are left out, and the places behind the others' get -1; a bin more than
// experts counts nothing and is where they begin.
constexpr int kPlanWaves = 16;
static_assert(kMostExperts < 64 * kPlanWaves, "a thread for each bin");

// the expert of a slot, -1: none here
__device__ __forceinline__ int bin_of(const PlanLaunch &a, int64_t slot)
{
    const uint32_t e = (uint32_t)a.ids[slot] - (uint32_t)a.first;
    return e < (uint32_t)a.E ? (int)e : -1;
}

// Bins of the slots s, s + step, ... below `to` (kHeld of them at most; -1 behind), in one go; 0 <= s < a.S where
// any is read.
constexpr int kHeld = 4;
__device__ __forceinline__ void hold_bins(const PlanLaunch &a, int64_t s, int64_t step, int64_t to, int (&bin)[kHeld])
{
#pragma unroll
    for (int i = 0; i < kHeld; i++) bin[i] = -1;
    if (s >= to) return;
#pragma unroll
    for (int i = 0; i < kHeld; i++) {
        const int64_t at = s + i * step;
        const int b = bin_of(a, at < to ? at : s);
        bin[i] = at < to ? b : -1;
    }
}

// slots of each bin in each run
__global__ __launch_bounds__(64 * kPlanWaves)
void plan_count_kernel(const PlanLaunch a)
{
    __shared__ int count[kMostExperts + 1];
    for (int i = threadIdx.x; i <= a.E; i += 64 * kPlanWaves) count[i] = 0;
    __syncthreads();
    constexpr int64_t step = 64 * kPlanWaves;
    const int64_t from = (int64_t)blockIdx.x * a.run, to = from + a.run < a.S ? from + a.run : a.S;
    for (int64_t s = from; s < to; s += kHeld * step) {
        int bin[kHeld];
        hold_bins(a, s + threadIdx.x, step, to, bin);
#pragma unroll
        for (int i = 0; i < kHeld; i++)
            if (bin[i] >= 0) atomicAdd(&count[bin[i]], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= a.E; i += 64 * kPlanWaves) a.counts[(int64_t)blockIdx.x * (a.E + 1) + i] = count[i];
}

// Bound by chains of loads: a wave holds the bins of its first 256 slots from the count to the sort, and all
// threads share the counts of the runs.  Both launches in a captured loop, 160 thousand slots on 32 of 64 experts:
// 12.0 -> 7.7 us, half of that by leaving out the slots of no expert here, whose one bin took half of the
// additions; 1.6 million slots on 64: 21.7 -> 16.2.
__global__ __launch_bounds__(64 * kPlanWaves)
void plan_kernel(const PlanLaunch a)
{
    extern __shared__ int next[];                     // [wave][bin]: its count, then where its next slot goes
    __shared__ int named, sums[kPlanWaves], run_all[kMostExperts + 1], run_before[kMostExperts + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bins = a.E + 1;
    const int64_t part = a.run / kPlanWaves;          // a multiple of 64
    const int64_t from = (int64_t)blockIdx.x * a.run + wave * part;
    const int64_t to = from + part < a.S ? from + part : a.S, rest = from + kHeld * 64;
    int held[kHeld];
    hold_bins(a, from + lane, 64, to, held);
    for (int i = tid; i < kPlanWaves * bins; i += 64 * kPlanWaves) next[i] = 0;
    for (int i = tid; i < bins; i += 64 * kPlanWaves) run_all[i] = run_before[i] = 0;
    __syncthreads();
    if (a.runs > 1) {
        // slots of a bin in all runs, and in the runs before this one: a group of whole waves has a thread for
        // every bin, and the groups deal the runs out
        const int waves = (bins + 63) >> 6, groups = kPlanWaves / waves, group = wave / waves;
        const int bin = tid - group * waves * 64;
        if (group < groups && bin < bins) {
            int all = 0, before = 0;
#pragma unroll 4
            for (int b = group; b < (int)a.runs; b += groups) {
                const int c = a.counts[(int64_t)b * bins + bin];
                all += c;
                before += b < (int)blockIdx.x ? c : 0;
            }
            atomicAdd(&run_all[bin], all);
            atomicAdd(&run_before[bin], before);
        }
    }
#pragma unroll
    for (int i = 0; i < kHeld; i++)
        if (held[i] >= 0) atomicAdd(&next[wave * bins + held[i]], 1);
    for (int64_t s = rest + lane; s < to; s += 64) {
        const int bin = bin_of(a, s);
        if (bin >= 0) atomicAdd(&next[wave * bins + bin], 1);
    }
    __syncthreads();

    int all = 0;
    if (tid < bins) {
        if (a.runs == 1) {
            for (int w = 0; w < kPlanWaves; w++) all += next[w * bins + tid];
        } else {
            all = run_all[tid];
        }
    }
    const int upto = wave_scan(all);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - all;
    for (int w = 0; w < wave; w++) at += sums[w];
    if (tid < bins) {
        if (blockIdx.x == 0) a.offsets[tid] = at;
        if (tid == a.E) named = at;
        at += run_before[tid];
        for (int w = 0; w < kPlanWaves; w++) {
            const int c = next[w * bins + tid];
            next[w * bins + tid] = at;
            at += c;
        }
    }
    __syncthreads();

#pragma unroll 1
    for (int64_t s0 = from; s0 < to; s0 += 64) {
        const int64_t s = s0 + lane;
        int bin = held[0];
        if (s0 < rest) {
#pragma unroll
            for (int i = 0; i + 1 < kHeld; i++) held[i] = held[i + 1];
        } else {
            bin = s < to ? bin_of(a, s) : -1;
        }
        const bool live = bin >= 0;
        uint64_t same = __builtin_amdgcn_ballot_w64(live);       // lanes of this lane's bin
        for (int bit = 0; bit < a.bin_bits; bit++) {
            const bool one = bin >> bit & 1;
            const uint64_t ones = __builtin_amdgcn_ballot_w64(one);
            same &= one ? ones : ~ones;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int *const place = next + wave * bins + (live ? bin : 0);
        int at = 0;
        if (live) at = *place + rank;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (live && rank == 0) *place = at + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        // within the rows even where another stream has changed the choices since they were counted
        if (live && (uint32_t)at < (uint64_t)a.S) a.rows[at] = (int)s;
    }
    // behind the experts' slots: -1
    for (int64_t s = from + lane; s < to; s += 64)
        if (s >= named) a.rows[s] = -1;
}

// ------------------------------------------------------------------------- weighted sum ----

template <int DT> __device__ __forceinline__ uint32_t round_to(float v);
template <> __device__ __forceinline__ uint32_t round_to<0>(float v) { return __bfloat16_as_ushort(__float2bfloat16(v)); }
template <> __device__ __forceinline__ uint32_t round_to<1>(float v) { return __half_as_ushort(__float2half(v)); }
template <> __device__ __forceinline__ uint32_t round_to<2>(float v) { return __float_as_uint(v); }

// 16 bytes of a row in one access, wherever the row begins: rows are element-aligned, and the hardware takes
// such an access at any address.  Elements past the row's end are neither read nor written.  PAST: read past the
// caches; chosen when the kernel is compiled, because the compiler makes one plain load of a choice at run time.
template <int DT>
struct Piece {
    typedef typename Elem<DT>::T T;
    static constexpr int V = 16 / (int)sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(V)));
    typedef Vec Loose __attribute__((aligned(sizeof(T))));
    T e[V];
    template <bool PAST>
    __device__ __forceinline__ void load(const T *p, int left)
    {
        if (left >= V) {
            Vec v;
            if constexpr (PAST) v = __builtin_nontemporal_load(reinterpret_cast<const Loose *>(p));
            else v = *reinterpret_cast<const Loose *>(p);
#pragma unroll
            for (int i = 0; i < V; i++) e[i] = v[i];
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) e[i] = i < left ? p[i] : (T)0;
        }
    }
    __device__ __forceinline__ void store(T *p, int left) const
    {
        if (left >= V) {
            Vec v;
#pragma unroll
            for (int i = 0; i < V; i++) v[i] = e[i];
            *reinterpret_cast<Loose *>(p) = v;
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i < left) p[i] = e[i];
        }
    }
};

// A wave takes 64 pieces of 16 bytes of one token's row; the rows of up to kAhead choices are requested
// before the first is used.  Rows that the last cache does not hold are read past the caches (8 rows a token, just
// written: 3000 tokens of 4096 FP32 88 -> 62 us, 6000 of 5376 bf16 126 -> 112, 19989 391 -> 387), others may still
// lie there (1500 tokens of 4096 FP32: 25.8 us, 26.6 past the caches; 512 of 5376 bf16 11.0 and 11.6).  Bound by
// HBM: 19989 tokens, 8 rows of 5376 bf16 with a residual 384 us on the same rows again, 5.6 TB/s.
constexpr int kCombineWaves = 4, kAhead = 8;

template <int DT, bool PAST>
__global__ __launch_bounds__(64 * kCombineWaves)
void combine_kernel(const CombineLaunch a)
{
    using P = Piece<DT>;
    typedef typename P::T T;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t task = blockIdx.x * (uint32_t)kCombineWaves + wave;
    const int64_t t = task / (uint32_t)a.pieces;
    if (t >= a.T) return;
    const int n = ((int)(task % (uint32_t)a.pieces) * 64 + lane) * P::V;
    const int left = a.N - n;
    if (left <= 0) return;
    float sum[P::V];
#pragma unroll
    for (int i = 0; i < P::V; i++) sum[i] = 0.0f;
    const int32_t *ids = a.ids + t * a.k;
    const float *weights = a.weights + t * a.k;
    const T *y = static_cast<const T *>(a.y) + t * a.k * a.ld_y + n;
    P res;
    if (a.residual) res.template load<false>(static_cast<const T *>(a.residual) + t * a.ld_res + n, left);
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
        P p[kAhead];
        bool here[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            here[j] = j0 + j < a.k && (uint32_t)ids[j0 + j] - (uint32_t)a.first < (uint32_t)a.E;
            if (here[j]) p[j].template load<PAST>(y + (j0 + j) * a.ld_y, left);
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++)
            if (here[j]) {
                const float w = weights[j0 + j];
#pragma unroll
                for (int i = 0; i < P::V; i++) sum[i] = fmaf(w, Elem<DT>::cvt(p[j].e[i]), sum[i]);
            }
    }
    P o;
#pragma unroll
    for (int i = 0; i < P::V; i++) {
        if (a.residual) sum[i] += Elem<DT>::cvt(res.e[i]);
        const uint32_t b = round_to<DT>(sum[i]);
        if constexpr (DT == 2) o.e[i] = __uint_as_float(b);
        else o.e[i] = (T)b;
    }
    o.store(static_cast<T *>(a.out) + t * a.ld_out + n, left);
}

template <int DT>
hipError_t launch_combine_of(CombineLaunch a, hipStream_t st)
{
    constexpr int cols = 64 * Piece<DT>::V;
    a.pieces = (a.N + cols - 1) / cols;
    const bool past = a.T * a.k > (int64_t)(256 << 20) / (int64_t)sizeof(typename Elem<DT>::T) / a.N;
    const int64_t waves = a.T * a.pieces;
    const dim3 grid((unsigned)((waves + kCombineWaves - 1) / kCombineWaves)), threads(64 * kCombineWaves);
    if (past) hipLaunchKernelGGL((combine_kernel<DT, true>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((combine_kernel<DT, false>), grid, threads, 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_route_experts(RouteLaunch a, int dtype, hipStream_t st)
{
    a.lanes_lg = 0;
    while ((2 << a.lanes_lg) * a.G <= 64) a.lanes_lg++;
    a.group_size = a.E / a.G;
    a.group_factor = ((1u << 20) + a.group_size - 1) / a.group_size;
    switch (dtype) {
    case 0: return launch_route_of<0>(a, st);
    case 1: return launch_route_of<1>(a, st);
    case 2: return launch_route_of<2>(a, st);
    default: return hipErrorInvalidValue;
    }
}

// One workgroup up to 4096 slots, above runs of 1024 (8192 slots: 6.6 us, 9.1 by one workgroup) and, where the
// counts of the runs before become the longer part, of 2048 for few experts (160 thousand slots, 32 experts:
// 7.7 us, 8.6 with 4096) and of 4096 for many (512 experts: 12.8, 15.1 with 2048); at most 256 runs.
void plan_runs(int64_t S, int64_t E, int64_t &runs, int64_t &run)
{
    constexpr int64_t step = 64 * kPlanWaves;
    if (S < 1) S = 1;
    const int64_t length = S <= 65536 ? 1024 : E <= 128 ? 2048 : 4096;
    runs = S <= kOneRun ? 1 : (S + length - 1) / length;
    if (runs > 256) runs = 256;
    run = ((S + runs - 1) / runs + step - 1) / step * step;
    runs = (S + run - 1) / run;
}

hipError_t launch_experts_plan(PlanLaunch a, hipStream_t st)
{
    plan_runs(a.S, a.E, a.runs, a.run);
    a.bin_bits = 0;
    while ((1 << a.bin_bits) <= a.E) a.bin_bits++;
    const dim3 grid((unsigned)a.runs), threads(64 * kPlanWaves);
    if (a.runs > 1) {
        hipLaunchKernelGGL(plan_count_kernel, grid, threads, 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(plan_kernel, grid, threads, (size_t)kPlanWaves * (a.E + 1) * sizeof(int), st, a);
    return hipGetLastError();
}

hipError_t launch_experts_combine(const CombineLaunch &a, int dtype, hipStream_t st)
{
    switch (dtype) {
    case 0: return launch_combine_of<0>(a, st);
    case 1: return launch_combine_of<1>(a, st);
    case 2: return launch_combine_of<2>(a, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
