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

__device__ __forceinline__ double shfl_xor_f64(double v, int m) { return __shfl_xor(v, m); }

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v += shfl_xor_f64(v, m);
    return v;
}

// One wave a token; lane l holds experts l, l + 64, ...  Scores are computed in FP64, so that which of
// two experts is chosen does not turn on a rounding; without a bias the logits order the experts as
// the scores do, and only the chosen ones' scores are computed.  k times the wave's largest key, the
// lowest expert where several have it, is taken and struck out.
constexpr int kRouteWaves = 4;

template <int DT, int NE>
__global__ __launch_bounds__(64 * kRouteWaves)
void route_kernel(const RouteLaunch a)
{
    extern __shared__ double lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t = (int64_t)blockIdx.x * kRouteWaves + wave;
    if (t >= a.T) return;
    const auto *row = static_cast<const typename Elem<DT>::T *>(a.logits) + t * a.ld;

    float l[NE];
    uint64_t key[NE];
    double score[NE] = {};
    uint32_t top = 0;
    bool valid[NE];
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = 64 * i + lane;
        l[i] = e < a.E ? Elem<DT>::cvt(row[e]) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        valid[i] = l[i] > -INFINITY;                  // neither -inf nor NaN
        const uint32_t b = __float_as_uint(l[i]), o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
        if (valid[i] && o > top) top = o;
    }
    top = wave_max(top);
    const float most = __uint_as_float(top ^ (top >> 31 ? 0x80000000u : 0xFFFFFFFFu));
    // exp(l - most), 1 where they are equal (infinite or not)
    auto power = [&](float x) { return x == most ? 1.0 : exp((double)x - (double)most); };
    auto sigmoid = [&](float x) { return 1.0 / (1.0 + exp(-(double)x)); };

    const bool grouped = a.top_groups < a.G;
    const bool all_scores = a.bias || (grouped && a.group_sum == 2);
    double norm = 1.0;                                // softmax: 1 / sum of the powers
    if (!a.sigmoid && (all_scores || !a.renorm)) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NE; i++) {
            score[i] = valid[i] ? power(l[i]) : 0.0;
            sum += score[i];
        }
        norm = 1.0 / wave_sum(sum);
    }
#pragma unroll
    for (int i = 0; i < NE; i++) {
        const int e = 64 * i + lane;
        double v = (double)l[i];
        if (all_scores) {
            score[i] = !valid[i] ? 0.0 : a.sigmoid ? sigmoid(l[i]) : score[i] * norm;
            if (a.bias) v = score[i] + (double)(valid[i] ? a.bias[e] : 0.0f);
        }
        valid[i] = valid[i] && v > -INFINITY;
        key[i] = valid[i] ? ordered(v) : 0;
        if (grouped) {
            if (a.group_sum == 2 && !a.bias) v = score[i];
            if (e < a.E) lds[wave * a.E + e] = valid[i] ? v : -INFINITY;
        }
    }
    if (grouped) {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        // 2^lanes_lg lanes a group: its largest and second largest value
        const int size = a.E / a.G, per = 1 << a.lanes_lg, g = lane >> a.lanes_lg;
        double b1 = -INFINITY, b2 = -INFINITY;
        if (g < a.G)
            for (int x = lane & (per - 1); x < size; x += per) {
                const double v = lds[wave * a.E + g * size + x];
                b2 = fmax(b2, fmin(b1, v));
                b1 = fmax(b1, v);
            }
        for (int m = 1; m < per; m <<= 1) {
            const double o1 = shfl_xor_f64(b1, m), o2 = shfl_xor_f64(b2, m);
            b2 = fmax(fmax(b2, o2), fmin(b1, o1));
            b1 = fmax(b1, o1);
        }
        const double v = a.group_sum == 2 && b2 > -INFINITY ? b1 + b2 : b1;
        int better = 0;                               // groups that come before this one
        for (int o = 0; o < a.G; o++) {
            const double w = __shfl(v, o << a.lanes_lg);
            better += w > v || (w == v && o < g);
        }
        const uint64_t kept = __builtin_amdgcn_ballot_w64(g < a.G && better < a.top_groups);
#pragma unroll
        for (int i = 0; i < NE; i++) {
            const int e = 64 * i + lane;
            if (e < a.E && !(kept >> ((e / size) << a.lanes_lg) & 1)) key[i] = 0;
        }
    }

    int id = -1;                                      // lane j: choice j
    float chosen = 0.0f;
    double s = 0.0;
    for (int j = 0; j < a.k; j++) {
        uint64_t best = key[0];
        int at = 0;
        float bl = l[0];
        double bs = score[0];
#pragma unroll
        for (int i = 1; i < NE; i++)
            if (key[i] > best) { best = key[i]; at = i; bl = l[i]; bs = score[i]; }
        const uint32_t hi = wave_max((uint32_t)(best >> 32));
        if (hi == 0) break;                           // none left (a number's key has a bit above)
        bool mine = (uint32_t)(best >> 32) == hi;
        const uint32_t lo = wave_max(mine ? (uint32_t)best : 0u);
        mine = mine && (uint32_t)best == lo;
        const uint32_t inv = wave_max(mine ? ~(uint32_t)(64 * at + lane) : 0u);
        const int e = (int)~inv, from = e & 63;
#pragma unroll
        for (int i = 0; i < NE; i++)
            if (64 * i + lane == e) key[i] = 0;
        const float wl = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(bl), from));
        const uint64_t bits = (uint64_t)__double_as_longlong(bs);
        const uint32_t s0 = __builtin_amdgcn_readlane((uint32_t)bits, from);
        const uint32_t s1 = __builtin_amdgcn_readlane((uint32_t)(bits >> 32), from);
        if (lane == j) {
            id = e;
            chosen = wl;
            s = __longlong_as_double((int64_t)((uint64_t)s1 << 32 | s0));
        }
    }
    if (!all_scores) s = id < 0 ? 0.0 : a.sigmoid ? sigmoid(chosen) : power(chosen) * norm;
    if (id < 0) s = 0.0;
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
// order; a bin more than experts takes the slots of no expert here.
constexpr int kPlanWaves = 16;
static_assert(kMostExperts < 64 * kPlanWaves, "a thread for each bin");

__device__ __forceinline__ int bin_of(const PlanLaunch &a, int64_t slot)
{
    const uint32_t e = (uint32_t)a.ids[slot] - (uint32_t)a.first;
    return e < (uint32_t)a.E ? (int)e : a.E;
}

// slots of each bin in each run
__global__ __launch_bounds__(64 * kPlanWaves)
void plan_count_kernel(const PlanLaunch a)
{
    __shared__ int count[kMostExperts + 1];
    for (int i = threadIdx.x; i <= a.E; i += 64 * kPlanWaves) count[i] = 0;
    __syncthreads();
    const int64_t from = (int64_t)blockIdx.x * a.run, to = from + a.run < a.S ? from + a.run : a.S;
    for (int64_t s = from + threadIdx.x; s < to; s += 64 * kPlanWaves) atomicAdd(&count[bin_of(a, s)], 1);
    __syncthreads();
    for (int i = threadIdx.x; i <= a.E; i += 64 * kPlanWaves) a.counts[(int64_t)blockIdx.x * (a.E + 1) + i] = count[i];
}

__global__ __launch_bounds__(64 * kPlanWaves)
void plan_kernel(const PlanLaunch a)
{
    extern __shared__ int next[];                     // [wave][bin]: its count, then where its next slot goes
    __shared__ int sums[kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int bins = a.E + 1;
    for (int i = tid; i < kPlanWaves * bins; i += 64 * kPlanWaves) next[i] = 0;
    __syncthreads();
    const int64_t part = a.run / kPlanWaves;          // a multiple of 64
    const int64_t from = (int64_t)blockIdx.x * a.run + wave * part;
    const int64_t to = from + part < a.S ? from + part : a.S;
    for (int64_t s = from + lane; s < to; s += 64) atomicAdd(&next[wave * bins + bin_of(a, s)], 1);
    __syncthreads();

    // thread e: slots of bin e in all runs, and in the runs before this one
    int all = 0, before = 0;
    if (tid < bins) {
        if (a.runs == 1) {
            for (int w = 0; w < kPlanWaves; w++) all += next[w * bins + tid];
        } else {
#pragma unroll 8
            for (int b = 0; b < (int)a.runs; b++) {
                const int c = a.counts[(int64_t)b * bins + tid];
                all += c;
                before += b < (int)blockIdx.x ? c : 0;
            }
        }
    }
    const int upto = wave_scan(all);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int at = upto - all;
    for (int w = 0; w < wave; w++) at += sums[w];
    if (tid < bins) {
        if (blockIdx.x == 0) a.offsets[tid] = at;     // the slots of no expert come last
        at += before;
        for (int w = 0; w < kPlanWaves; w++) {
            const int c = next[w * bins + tid];
            next[w * bins + tid] = at;
            at += c;
        }
    }
    __syncthreads();

    for (int64_t s0 = from; s0 < to; s0 += 64) {
        const int64_t s = s0 + lane;
        const bool live = s < to;
        const int bin = live ? bin_of(a, s) : 0;
        uint64_t same = __builtin_amdgcn_ballot_w64(live);       // lanes of this lane's bin
        for (int bit = 0; bit < a.bin_bits; bit++) {
            const bool one = bin >> bit & 1;
            const uint64_t ones = __builtin_amdgcn_ballot_w64(one);
            same &= one ? ones : ~ones;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        int *const place = next + wave * bins + bin;
        int at = 0;
        if (live) at = *place + rank;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (live && rank == 0) *place = at + __popcll(same);
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        if (live) a.rows[at] = bin < a.E ? (int)s : -1;
    }
}

// ------------------------------------------------------------------------- weighted sum ----

template <int DT> __device__ __forceinline__ uint32_t round_to(float v);
template <> __device__ __forceinline__ uint32_t round_to<0>(float v) { return __bfloat16_as_ushort(__float2bfloat16(v)); }
template <> __device__ __forceinline__ uint32_t round_to<1>(float v) { return __half_as_ushort(__float2half(v)); }
template <> __device__ __forceinline__ uint32_t round_to<2>(float v) { return __float_as_uint(v); }

// V elements of a row in one access
template <int DT, int V>
struct Piece {
    static constexpr int ES = DT == 2 ? 4 : 2, B = V * ES;
    typedef typename Elem<DT>::T T;
    typedef T Vec __attribute__((ext_vector_type(V)));
    T e[V];
    __device__ __forceinline__ void load(const T *p, int left)
    {
        if (left >= V) {
            if constexpr (V == 1) e[0] = *p;
            else {
                const Vec v = *reinterpret_cast<const Vec *>(p);
#pragma unroll
                for (int i = 0; i < V; i++) e[i] = v[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i++) e[i] = i < left ? p[i] : (T)0;
        }
    }
    __device__ __forceinline__ void store(T *p, int left) const
    {
        if (left >= V) {
            if constexpr (V == 1) *p = e[0];
            else {
                Vec v;
#pragma unroll
                for (int i = 0; i < V; i++) v[i] = e[i];
                *reinterpret_cast<Vec *>(p) = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                if (i < left) p[i] = e[i];
        }
    }
};

// Threads take V columns of one token; the rows of up to kAhead choices are requested before the first
// is used.  Bound by HBM.
constexpr int kCombineThreads = 256, kAhead = 8;

template <int DT, int V>
__global__ __launch_bounds__(kCombineThreads)
void combine_kernel(const CombineLaunch a)
{
    typedef typename Elem<DT>::T T;
    const int64_t t = blockIdx.x / (uint32_t)a.pieces;
    const int n = ((int)(blockIdx.x % (uint32_t)a.pieces) * kCombineThreads + (int)threadIdx.x) * V;
    const int left = a.N - n;
    if (left <= 0) return;
    float sum[V];
#pragma unroll
    for (int i = 0; i < V; i++) sum[i] = 0.0f;
    const int32_t *ids = a.ids + t * a.k;
    const float *weights = a.weights + t * a.k;
    const T *y = static_cast<const T *>(a.y) + t * a.k * a.ld_y + n;
    Piece<DT, V> res;
    if (a.residual) res.load(static_cast<const T *>(a.residual) + t * a.ld_res + n, left);
    for (int j0 = 0; j0 < a.k; j0 += kAhead) {
        Piece<DT, V> p[kAhead];
        bool here[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++) {
            here[j] = j0 + j < a.k && (uint32_t)ids[j0 + j] - (uint32_t)a.first < (uint32_t)a.E;
            if (here[j]) p[j].load(y + (j0 + j) * a.ld_y, left);
        }
#pragma unroll
        for (int j = 0; j < kAhead; j++)
            if (here[j]) {
                const float w = weights[j0 + j];
#pragma unroll
                for (int i = 0; i < V; i++) sum[i] = fmaf(w, Elem<DT>::cvt(p[j].e[i]), sum[i]);
            }
    }
    Piece<DT, V> o;
#pragma unroll
    for (int i = 0; i < V; i++) {
        if (a.residual) sum[i] += Elem<DT>::cvt(res.e[i]);
        const uint32_t b = round_to<DT>(sum[i]);
        if constexpr (DT == 2) o.e[i] = __uint_as_float(b);
        else o.e[i] = (T)b;
    }
    o.store(static_cast<T *>(a.out) + t * a.ld_out + n, left);
}

template <int DT, int V>
hipError_t launch_combine_of(CombineLaunch a, hipStream_t st)
{
    a.pieces = (a.N + kCombineThreads * V - 1) / (kCombineThreads * V);
    hipLaunchKernelGGL((combine_kernel<DT, V>), dim3((unsigned)(a.T * a.pieces)), dim3(kCombineThreads), 0, st, a);
    return hipGetLastError();
}

// elements that every row's start allows in one access of at most 16 bytes
int combine_elements(const CombineLaunch &a, int es)
{
    uintptr_t bits = (uintptr_t)a.y | (uintptr_t)a.out | (uintptr_t)(a.ld_y * es) | (uintptr_t)(a.ld_out * es);
    if (a.residual) bits |= (uintptr_t)a.residual | (uintptr_t)(a.ld_res * es);
    const int bytes = bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : bits % 4 == 0 ? 4 : 2;
    return bytes / es;
}

template <int DT>
hipError_t launch_combine_dt(const CombineLaunch &a, hipStream_t st)
{
    switch (combine_elements(a, DT == 2 ? 4 : 2)) {
    case 1: return launch_combine_of<DT, 1>(a, st);
    case 2: return launch_combine_of<DT, 2>(a, st);
    case 4: return launch_combine_of<DT, 4>(a, st);
    default:
        if constexpr (DT == 2) return hipErrorInvalidValue;
        else return launch_combine_of<DT, 8>(a, st);
    }
}

}  // namespace

hipError_t launch_route_experts(RouteLaunch a, int dtype, hipStream_t st)
{
    a.lanes_lg = 0;
    while ((2 << a.lanes_lg) * a.G <= 64) a.lanes_lg++;
    switch (dtype) {
    case 0: return launch_route_of<0>(a, st);
    case 1: return launch_route_of<1>(a, st);
    case 2: return launch_route_of<2>(a, st);
    default: return hipErrorInvalidValue;
    }
}

// Runs of 2048 slots above 8192, so that a clip's 160 thousand fill a third of the device; at most 256
// runs, whose counts every workgroup adds up.
void plan_runs(int64_t S, int64_t &runs, int64_t &run)
{
    constexpr int64_t step = 64 * kPlanWaves;
    if (S < 1) S = 1;
    runs = S <= 8192 ? 1 : (S + 2047) / 2048;
    if (runs > 256) runs = 256;
    run = ((S + runs - 1) / runs + step - 1) / step * step;
    runs = (S + run - 1) / run;
}

hipError_t launch_experts_plan(PlanLaunch a, hipStream_t st)
{
    plan_runs(a.S, a.runs, a.run);
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
    case 0: return launch_combine_dt<0>(a, st);
    case 1: return launch_combine_dt<1>(a, st);
    case 2: return launch_combine_dt<2>(a, st);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace convrot
