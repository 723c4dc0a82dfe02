// C ABI of the rotated W8A8 NVFP4 linear layer: argument validation, device checks,
// launch configuration and the bounded-staging layer orchestration.
//
// Layer orchestration (ComfyUI Turing Utils README, "Load ConvRot DiT ..." bullet):
// the activation is prepared once; the weight is prepared in chunks of output rows into
// call-local S8 tiles of bounded size (two tiles alternate), each chunk followed by the
// GEMM that writes its column band of the output; with a second stream and several
// chunks, the preparation of chunk c+1 runs beside the GEMM of chunk c, ordered by
// producer/consumer events.  Short batches skip the S8 weight altogether: the GEMM decodes
// the weight blocks itself (decode-inside-GEMM).  Chunking, streams and the path taken
// change no value.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/convrot.h"
#include "kernels.hpp"

namespace {

constexpr int kMaxDevices = 64;
std::atomic<int> g_arch_ok[kMaxDevices];   // 0 unknown, 1 gfx950, 2 other (read-only cache)

cr_status current_device_ok()
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return CR_ERR_NO_DEVICE;
    }
    int s = g_arch_ok[dev].load(std::memory_order_relaxed);
    if (s == 0) {
        hipDeviceProp_t p;
        if (hipGetDeviceProperties(&p, dev) != hipSuccess) {
            (void)hipGetLastError();
            return CR_ERR_NO_DEVICE;
        }
        s = (std::strncmp(p.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
        g_arch_ok[dev].store(s, std::memory_order_relaxed);
    }
    return s == 1 ? CR_OK : CR_ERR_NO_DEVICE;
}

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int64_t elem_size(cr_dtype d)
{
    switch (d) {
    case CR_BF16: case CR_FP16: return 2;
    case CR_FP32: case CR_I32: return 4;
    default: return 0;
    }
}

inline cr_status from_hip(hipError_t e) { return e == hipSuccess ? CR_OK : CR_ERR_LAUNCH; }

constexpr int64_t kMaxRows = 0x7fffffff;

inline int64_t pad256(int64_t k) { return ((k + 255) / 256) * 256; }

cr_status check_flags(uint32_t flags)
{
    return (flags & ~(uint32_t)(CR_FLAG_FORCE_TWO_PASS | CR_FLAG_BLOCK_TRANSPOSED)) ? CR_ERR_INVALID_ARG : CR_OK;
}

cr_status check_act(const void *x, cr_dtype dt, int64_t ld_x, int64_t M, int64_t K, int64_t cols,
                    int8_t *x_s8, int64_t ld_s8, float *x_scale, uint32_t flags)
{
    if (M > 0 && (!x || !x_s8 || !x_scale)) return CR_ERR_INVALID_ARG;   // M = 0: nothing is read or written
    if (dt != CR_BF16 && dt != CR_FP16 && dt != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || K < 1 || M > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_x < cols || ld_s8 < kp) return CR_ERR_INVALID_ARG;
    const int64_t es = elem_size(dt);
    if (!aligned(x, 16) || (ld_x * es) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(x_s8, 16) || ld_s8 % 16 != 0 || !aligned(x_scale, 4)) return CR_ERR_MISALIGNED;
    return CR_OK;
}

cr_status check_weight(const uint8_t *w_fp4, int64_t ld_fp4, const uint8_t *w_sf, int64_t ld_sf,
                       const float *g, int64_t n_rows, int64_t K, int8_t *w_s8, int64_t ld_s8,
                       float *w_scale, uint32_t flags)
{
    if (n_rows > 0 && (!w_fp4 || !w_sf || !g || !w_s8 || !w_scale)) return CR_ERR_INVALID_ARG;
    if (n_rows < 0 || K < 1 || n_rows > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_fp4 < (K + 1) / 2 || ld_sf < (K + 15) / 16 || ld_s8 < kp) return CR_ERR_INVALID_ARG;
    if (!aligned(w_fp4, 16) || ld_fp4 % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(g, 4) || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
    if (!aligned(w_s8, 16) || ld_s8 % 16 != 0) return CR_ERR_MISALIGNED;
    return CR_OK;
}

cr_status check_gemm(const int8_t *a, int64_t lda, const float *sa, const int8_t *b, int64_t ldb,
                     const float *sb, int64_t M, int64_t N, int64_t K_pad, void *c, cr_dtype cdt,
                     int64_t ldc)
{
    if ((M > 0 && !a) || (N > 0 && !b) || (M > 0 && N > 0 && !c)) return CR_ERR_INVALID_ARG;
    if (cdt != CR_BF16 && cdt != CR_FP16 && cdt != CR_FP32 && cdt != CR_I32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (cdt != CR_I32 && ((M > 0 && !sa) || (N > 0 && !sb))) return CR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K_pad < 1 || K_pad % 256 != 0) return CR_ERR_INVALID_ARG;
    if (M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    // one workgroup of 512 threads per 256 x 256 tile; a dispatch counts work-items in 32 bits
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (K_pad > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (lda < K_pad || ldb < K_pad || ldc < N) return CR_ERR_INVALID_ARG;
    if (!aligned(a, 16) || !aligned(b, 16) || lda % 16 != 0 || ldb % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(c, (size_t)elem_size(cdt))) return CR_ERR_MISALIGNED;
    if ((sa && !aligned(sa, 4)) || (sb && !aligned(sb, 4))) return CR_ERR_MISALIGNED;
    return CR_OK;
}

cr_status check_fused(const int8_t *a_s8, int64_t lda, const float *a_scale, const uint8_t *w_fp4,
                      int64_t ld_fp4, const uint8_t *w_sf, int64_t ld_sf, const float *g, const float *w_amax,
                      const float *bias, int64_t M, int64_t N, int64_t K, void *c, cr_dtype c_dtype, int64_t ldc,
                      uint32_t flags)
{
    if ((M > 0 && !a_s8) || (N > 0 && (!w_fp4 || !w_sf || !g)) || (M > 0 && N > 0 && !c)) return CR_ERR_INVALID_ARG;
    if (c_dtype != CR_BF16 && c_dtype != CR_FP16 && c_dtype != CR_FP32 && c_dtype != CR_I32)
        return CR_ERR_UNSUPPORTED_DTYPE;
    if (c_dtype != CR_I32 && M > 0 && !a_scale) return CR_ERR_INVALID_ARG;
    if (bias && c_dtype == CR_I32) return CR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if ((M + 127) / 128 > 65535) return CR_ERR_TOO_LARGE;
    if ((N + 31) / 32 > (int64_t)(UINT32_MAX / 256)) return CR_ERR_TOO_LARGE;   // 32-bit work-item count
    if (lda < kp || ld_fp4 < (K + 1) / 2 || ld_sf < (K + 15) / 16 || ldc < N) return CR_ERR_INVALID_ARG;
    if (!aligned(a_s8, 16) || lda % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(w_fp4, 16) || ld_fp4 % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(g, 4) || (w_amax && !aligned(w_amax, 4))) return CR_ERR_MISALIGNED;
    if ((a_scale && !aligned(a_scale, 4)) || (bias && !aligned(bias, 4))) return CR_ERR_MISALIGNED;
    if (!aligned(c, (size_t)elem_size(c_dtype))) return CR_ERR_MISALIGNED;
    return CR_OK;
}

// Batches of at most this many activation rows run the layer with the weight decoded
// inside the GEMM (cr_gemm_nvfp4_fused, row maxima from its own first pass) instead of
// staging S8 weight tiles: with so few rows the decode dominates either way, and the
// staged path adds the S8 write and read of the whole weight and a GEMM with few tiles.
constexpr int64_t kFusedMaxRows = 64;

// Workspace layout of cr_linear_nvfp4 (every region 256-byte aligned):
//   staged: x_s8 [M, K_pad] | x_scale [M] | tile0 [R, K_pad] | tscale0 [R] | tile1 | tscale1
//   fused:  x_s8 [M, K_pad] | x_scale [M]
struct LayerPlan {
    bool fused;
    int64_t K_pad, R, nchunks;
    size_t off_xscale, off_tile[2], off_tscale[2], bytes;
};

inline size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

std::atomic<int> g_cus[kMaxDevices];       // 0 unknown (asked for once a device: 0.15 us a call)

int current_cus()
{
    int dev = -1, cus = 0;
    if (hipGetDevice(&dev) == hipSuccess && dev >= 0 && dev < kMaxDevices &&
        (cus = g_cus[dev].load(std::memory_order_relaxed)) > 0)
        return cus;
    if (dev < 0 || hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) {
        (void)hipGetLastError();
        return 256;
    }
    if (dev < kMaxDevices) g_cus[dev].store(cus, std::memory_order_relaxed);
    return cus;
}

// Rows per weight chunk, a multiple of the GEMM tile height.  The chunks' GEMMs run one
// after another, so each pays for whole rounds of workgroups over the CUs: a GEMM of
// t tiles takes ceil(t / cus) rounds.
// * When the tile bound forces several chunks, the chunk height within the bound is the
//   one whose GEMMs need the fewest rounds in total (the tallest of those on a tie).  With
//   M = 19989 (79 tile rows) and a 16 MiB bound on K_pad = 14336, 1024-row chunks would be
//   316-tile GEMMs of two rounds each (11 rounds for 5376 rows); 768-row chunks are
//   237-tile GEMMs of one round (7 rounds, as many as one unchunked GEMM).
// * When the whole weight fits one chunk it is still split in two whenever the two GEMMs
//   together need no more rounds than one GEMM would: with a second stream the second
//   chunk's preparation can then overlap the first chunk's GEMM, and staged serially the
//   split costs nothing (QKV at M = 19989: 1.93-1.95 ms for the two GEMMs against 1.94 ms
//   for one over the whole weight, same operands).
int64_t plan_rows(int64_t M, int64_t N, int64_t K_pad, size_t max_tile_bytes, int cus)
{
    const int64_t T = convrot::kGemmTileRows;
    int64_t kmax = (int64_t)(max_tile_bytes / (size_t)K_pad) / T;   // tile rows per chunk
    if (kmax < 1) kmax = 1;
    const int64_t tiles_n = (N + T - 1) / T;
    const int64_t tiles_m = (M + convrot::kGemmTileCols - 1) / convrot::kGemmTileCols;
    auto rounds = [&](int64_t tiles) { return (tiles + cus - 1) / cus; };
    if (kmax < tiles_n) {                               // chunked by the bound
        int64_t best_k = kmax, best = -1;
        for (int64_t k = kmax; k >= 1 && kmax - k < 4096; k--) {   // host time stays bounded
            const int64_t rem = tiles_n % k;
            const int64_t r = (tiles_n / k) * rounds(tiles_m * k) + (rem ? rounds(tiles_m * rem) : 0);
            if (best < 0 || r < best) { best = r; best_k = k; }
        }
        return best_k * T;
    }
    if (tiles_n < 2) return tiles_n * T;
    const int64_t t0 = (tiles_n + 1) / 2, t1 = tiles_n - t0;
    if (rounds(tiles_m * t0) + rounds(tiles_m * t1) <= rounds(tiles_m * tiles_n)) return t0 * T;
    return tiles_n * T;
}

LayerPlan plan_layer(int64_t M, int64_t N, int64_t K, size_t max_tile_bytes)
{
    LayerPlan p{};
    if (max_tile_bytes == 0) max_tile_bytes = CR_DEFAULT_MAX_TILE_BYTES;
    p.K_pad = pad256(K);
    if (M == 0 || N == 0) return p;                  // empty: no chunks, no workspace
    if (M <= kFusedMaxRows) {
        p.fused = true;
        p.off_xscale = up256((size_t)M * (size_t)p.K_pad);
        p.bytes = up256(p.off_xscale + (size_t)M * 4);
        return p;
    }
    p.R = plan_rows(M, N, p.K_pad, max_tile_bytes, current_cus());
    p.nchunks = (N + p.R - 1) / p.R;
    size_t off = up256((size_t)M * (size_t)p.K_pad);
    p.off_xscale = off;
    off = up256(off + (size_t)M * 4);
    const int ntiles = p.nchunks > 1 ? 2 : 1;
    for (int t = 0; t < 2; t++) {
        p.off_tile[t] = off;
        p.off_tscale[t] = up256(off + (size_t)p.R * (size_t)p.K_pad);
        if (t < ntiles) off = up256(p.off_tscale[t] + (size_t)p.R * 4);
    }
    p.bytes = off;
    return p;
}

// Events that order the staging stream against the main stream.  A layer call takes one
// set from a per-device pool and returns it once its work is enqueued: a wait enqueued on a
// stream refers to the event's most recent record at the time of the wait, so a set can be
// recorded again by the next call (on this thread or another) while earlier work is still
// in flight.  Sets are created on first need (as many as there are concurrent callers) and
// kept until the process ends; the pool is guarded by a mutex.
struct EventSet {
    hipEvent_t ev[5] = {nullptr, nullptr, nullptr, nullptr, nullptr};
};

std::mutex g_event_mu;
std::vector<EventSet *> g_event_pool[kMaxDevices];

class PooledEvents {
public:
    explicit PooledEvents(bool want)
    {
        if (!want) return;
        if (hipGetDevice(&dev_) != hipSuccess || dev_ < 0 || dev_ >= kMaxDevices) {
            (void)hipGetLastError();
            dev_ = -1;
            return;
        }
        {
            std::lock_guard<std::mutex> lk(g_event_mu);
            auto &pool = g_event_pool[dev_];
            if (!pool.empty()) {
                set_ = pool.back();
                pool.pop_back();
                return;
            }
        }
        auto *s = new (std::nothrow) EventSet;
        if (!s) return;
        for (auto &e : s->ev)
            if (hipEventCreateWithFlags(&e, hipEventDisableTiming) != hipSuccess) {
                (void)hipGetLastError();
                for (auto &d : s->ev)
                    if (d) (void)hipEventDestroy(d);
                delete s;
                return;
            }
        set_ = s;
    }
    ~PooledEvents()
    {
        if (!set_) return;
        std::lock_guard<std::mutex> lk(g_event_mu);
        g_event_pool[dev_].push_back(set_);
    }
    PooledEvents(const PooledEvents &) = delete;
    PooledEvents &operator=(const PooledEvents &) = delete;
    bool ok() const { return set_ != nullptr; }
    hipEvent_t operator[](int i) const { return set_->ev[i]; }

private:
    int dev_ = -1;
    EventSet *set_ = nullptr;
};

// Device scratch of cr_linear_nvfp4_noalloc: the layer's workspace for callers that cannot
// allocate.  One copy per GPU, created with the code object and held until the process
// ends.  In host code `scratch` names a host-side stand-in, not device memory: only the
// address that hipGetSymbolAddress returns for the current device may reach a kernel.
static __device__ __align__(256) int8_t scratch[CR_NOALLOC_SCRATCH_BYTES];

std::mutex g_scratch_mu;
void *g_scratch_ptr[kMaxDevices];   // device address of `scratch`, per device (guarded)

// The current device's copy of `scratch`, resolved on the first call on that device (with
// that device current) and kept.
cr_status scratch_for_current_device(void **out)
{
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return CR_ERR_NO_DEVICE;
    }
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void *p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) {
            (void)hipGetLastError();
            return CR_ERR_LAUNCH;
        }
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return CR_OK;
}

// The tile bound cr_linear_nvfp4_noalloc uses when the caller passes 0: the largest one for
// which the activation and two S8 weight tiles (with their scales) fit the scratch; 0 when
// not even the activation and two 256-row tiles fit.
size_t noalloc_tile_bound(int64_t M, int64_t K)
{
    const int64_t kp = pad256(K);
    const size_t act = up256((size_t)M * (size_t)kp) + up256((size_t)M * 4);
    if (act + 512 >= CR_NOALLOC_SCRATCH_BYTES) return 0;
    const size_t rem = CR_NOALLOC_SCRATCH_BYTES - act - 512;
    const int64_t T = convrot::kGemmTileRows;
    const int64_t rows = (int64_t)(rem / (2 * ((size_t)kp + 4))) / T * T;
    return rows < T ? 0 : (size_t)rows * (size_t)kp;
}

// ---- the 8-bit cache ----

constexpr int64_t kMaxHeads = 65535;

// what the two calls over the cache have in common; `needs_cache` false: no head reads or
// writes it.  Pointers are only needed when there are tokens.
cr_status check_kv8(cr_dtype dt, int64_t T, int64_t B, const int32_t *cu, const int32_t *kv_lens, int64_t Hq,
                    int64_t Hkv, int64_t D, const cr_kv8_cache *c, bool needs_cache)
{
    if (dt != CR_BF16 && dt != CR_FP16) return CR_ERR_UNSUPPORTED_DTYPE;
    if (T < 0 || B < 0 || T > kMaxRows || B > kMaxRows) return CR_ERR_INVALID_ARG;
    if (Hq < 0 || Hkv < 0 || Hq > kMaxHeads || Hkv > kMaxHeads || (D != 64 && D != 128)) return CR_ERR_INVALID_ARG;
    const bool any = T > 0 && B > 0;
    if (any && (!cu || !kv_lens)) return CR_ERR_INVALID_ARG;
    if (!aligned(cu, 4) || !aligned(kv_lens, 4)) return CR_ERR_MISALIGNED;
    if (!needs_cache) return CR_OK;
    if (!c) return CR_ERR_INVALID_ARG;
    if (c->n_pages < 0 || c->ld_table < 0) return CR_ERR_INVALID_ARG;
    if (c->ld_table > CR_KV8_MAX_PAGES || c->n_pages > kMaxRows) return CR_ERR_TOO_LARGE;
    if (any && (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->page_table)) return CR_ERR_INVALID_ARG;
    if (any && (c->n_pages < 1 || c->ld_table < 1)) return CR_ERR_INVALID_ARG;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        !aligned(c->page_table, 4))
        return CR_ERR_MISALIGNED;
    return CR_OK;
}

// rows [T, ld] of 16-bit elements holding `cols` of them
cr_status check_rows16(const void *p, int64_t ld, int64_t cols, bool any)
{
    if (any && !p) return CR_ERR_INVALID_ARG;
    if (ld < cols) return CR_ERR_INVALID_ARG;
    return (!aligned(p, 16) || ld % 8 != 0) ? CR_ERR_MISALIGNED : CR_OK;
}

convrot::Kv8Ptrs kv8_ptrs(const cr_kv8_cache *c)
{
    if (!c) return convrot::Kv8Ptrs{};
    return convrot::Kv8Ptrs{c->k, c->v, c->k_scale, c->v_scale, c->n_pages, c->page_table, c->ld_table};
}

// the attention's plan on the current device; false where its sizes are not a valid call's or
// exceed what the launch can count
bool attn_plan(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t Hq, int64_t Hkv, int64_t D,
               convrot::AttnPlan *p)
{
    if (T < 0 || B < 0 || max_q < 0 || max_kv < 0 || T > kMaxRows || B > kMaxRows || max_q > kMaxRows) return false;
    if (Hq < 1 || Hkv < 1 || Hq > kMaxHeads || Hq % Hkv != 0 || (D != 64 && D != 128)) return false;
    if (max_q > T) max_q = T;
    if (max_kv > CR_KV8_MAX_PAGES * CR_KV8_PAGE) max_kv = CR_KV8_MAX_PAGES * CR_KV8_PAGE;
    *p = convrot::plan_attn_kv8(T, B, max_q, max_kv, (int)Hq, (int)Hkv, (int)D, current_cus());
    return true;
}

// ---- a layer of experts ----

static_assert(CR_MAX_EXPERTS == convrot::kMostExperts && CR_MAX_CHOICES == convrot::kMostChoices &&
              CR_MAX_EXPERT_GROUPS == convrot::kMostGroups && CR_PLAN_SLOTS_IN_PLACE == convrot::kOneRun, "limits of the header and the kernels");

// tokens, choices and the experts here
cr_status check_slots(int64_t T, int64_t top_k, int64_t first, int64_t E)
{
    if (T < 0 || top_k < 1 || top_k > CR_MAX_CHOICES || E < 1 || E > CR_MAX_EXPERTS) return CR_ERR_INVALID_ARG;
    if (first < 0 || first > kMaxRows - E || T > kMaxRows / top_k) return CR_ERR_INVALID_ARG;
    return CR_OK;
}

bool is_float(cr_dtype d) { return d == CR_BF16 || d == CR_FP16 || d == CR_FP32; }

// one weight of every expert: packed rows, strides in bytes, scales and an optional bias
cr_status check_expert_weight(const uint8_t *w, int64_t ld, int64_t stride, const float *scale, const float *bias,
                              int64_t N, int64_t K_pad, bool needs_scale)
{
    if (N > 0 && (!w || (needs_scale && !scale))) return CR_ERR_INVALID_ARG;
    if (N < 0 || N > kMaxRows || K_pad < 1 || K_pad % 256 != 0) return CR_ERR_INVALID_ARG;
    if (K_pad > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld < K_pad / 2 || ld > kMaxRows || stride < N * ld) return CR_ERR_INVALID_ARG;
    if (!aligned(w, 16) || ld % 16 != 0 || stride % 16 != 0 || !aligned(scale, 4) || !aligned(bias, 4))
        return CR_ERR_MISALIGNED;
    return CR_OK;
}

cr_status check_experts_gemm(const int8_t *a, int64_t lda, const float *sa, int64_t M, const uint8_t *b, int64_t ldb,
                             int64_t stride, const float *sb, const float *bias, const int32_t *offsets,
                             const int32_t *rows, int64_t S, int64_t E, int64_t N, int64_t K_pad, int64_t gather,
                             const void *c, cr_dtype cdt, int64_t ldc, uint32_t flags)
{
    const bool swiglu = (flags & CR_FLAG_EXPERTS_SWIGLU) != 0, scatter = (flags & CR_FLAG_EXPERTS_SCATTER) != 0;
    if (!is_float(cdt) && cdt != CR_I32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (flags & ~(uint32_t)(CR_FLAG_EXPERTS_SCATTER | CR_FLAG_EXPERTS_SWIGLU)) return CR_ERR_INVALID_ARG;
    if (M < 0 || S < 0 || M > kMaxRows || S > kMaxRows || E < 1 || E > CR_MAX_EXPERTS) return CR_ERR_INVALID_ARG;
    if (gather < 0 || gather > CR_MAX_CHOICES) return CR_ERR_INVALID_ARG;
    if (cdt == CR_I32 && (swiglu || bias)) return CR_ERR_INVALID_ARG;
    if (swiglu && N % 2 != 0) return CR_ERR_INVALID_ARG;
    const bool any = S > 0 && N > 0 && M > 0;
    cr_status s = check_expert_weight(b, ldb, stride, sb, bias, N, K_pad, cdt != CR_I32);
    if (s != CR_OK) return s;
    if (lda < K_pad || ldc < (swiglu ? N / 2 : N)) return CR_ERR_INVALID_ARG;
    if (any && (!a || !offsets || !c || (cdt != CR_I32 && !sa))) return CR_ERR_INVALID_ARG;
    if (any && (gather > 0 || scatter) && !rows) return CR_ERR_INVALID_ARG;
    if (!aligned(a, 16) || lda % 16 != 0 || !aligned(sa, 4) || !aligned(offsets, 4) || !aligned(rows, 4))
        return CR_ERR_MISALIGNED;
    if (!aligned(c, (size_t)elem_size(cdt))) return CR_ERR_MISALIGNED;
    // 32-bit count of work-items
    if (any && convrot::experts_gemm_blocks(S, E, N) > convrot::kMostBlocks) return CR_ERR_TOO_LARGE;
    return CR_OK;
}

cr_status check_combine(const void *y, cr_dtype dt, int64_t ld_y, const float *weights, const int32_t *ids, int64_t T,
                        int64_t top_k, int64_t first, int64_t E, int64_t N, const void *residual, int64_t ld_res,
                        const void *out, int64_t ld_out)
{
    if (!is_float(dt)) return CR_ERR_UNSUPPORTED_DTYPE;
    cr_status s = check_slots(T, top_k, first, E);
    if (s != CR_OK) return s;
    if (N < 0 || N > kMaxRows || ld_y < N || ld_out < N || (residual && ld_res < N)) return CR_ERR_INVALID_ARG;
    if (T > 0 && N > 0 && (!y || !weights || !ids || !out)) return CR_ERR_INVALID_ARG;
    if (residual && residual == out && ld_res != ld_out) return CR_ERR_INVALID_ARG;
    const size_t es = (size_t)elem_size(dt);
    if (!aligned(y, es) || !aligned(residual, es) || !aligned(out, es) || !aligned(weights, 4) || !aligned(ids, 4))
        return CR_ERR_MISALIGNED;
    // workgroups of 256 threads with at least one column each
    if (T > 0 && (N + 255) / 256 > convrot::kMostBlocks / T) return CR_ERR_TOO_LARGE;
    return CR_OK;
}

size_t plan_bytes(int64_t S, int64_t E)
{
    int64_t runs, run;
    convrot::plan_runs(S, E, runs, run);
    return runs > 1 ? up256((size_t)runs * (size_t)(E + 1) * 4) : 0;
}

convrot::PlanLaunch plan_launch(const int32_t *ids, int64_t S, int64_t first, int64_t E, int32_t *offsets, int32_t *rows,
                                void *workspace)
{
    convrot::PlanLaunch p{};
    p.ids = ids; p.S = S; p.first = (int)first; p.E = (int)E; p.offsets = offsets; p.rows = rows;
    p.counts = static_cast<int32_t *>(workspace);
    return p;
}

convrot::ExpertsGemm experts_gemm(const int8_t *a, int64_t lda, const float *sa, int64_t M, const uint8_t *b, int64_t ldb,
                                  int64_t stride, const float *sb, const float *bias, const int32_t *offsets,
                                  const int32_t *rows, int64_t S, int64_t E, int64_t N, int64_t K_pad, int64_t gather,
                                  bool scatter, void *c, int64_t ldc)
{
    convrot::ExpertsGemm g{};
    g.A = a; g.lda = lda; g.sa = sa; g.M = (int)M; g.B = b; g.ldb = ldb; g.stride_b = stride; g.sb = sb; g.bias = bias;
    g.offsets = offsets; g.rows = rows; g.S = (int)S; g.E = (int)E; g.N = (int)N; g.K_pad = (int)K_pad;
    g.gather = (int)gather; g.scatter = scatter; g.C = c; g.ldc = ldc;
    return g;
}

convrot::CombineLaunch combine_launch(const void *y, int64_t ld_y, const float *weights, const int32_t *ids, int64_t T,
                                      int64_t top_k, int64_t first, int64_t E, int64_t N, const void *residual,
                                      int64_t ld_res, void *out, int64_t ld_out)
{
    convrot::CombineLaunch c{};
    c.y = y; c.ld_y = ld_y; c.weights = weights; c.ids = ids; c.T = T; c.k = (int)top_k; c.first = (int)first;
    c.E = (int)E; c.N = (int)N; c.residual = residual; c.ld_res = ld_res; c.out = out; c.ld_out = ld_out;
    return c;
}

constexpr int64_t kMostExpertCols = 1 << 28;     // columns of the layer's output: byte counts stay below 2^63

// Workspace of the layer of experts (every region 256-byte aligned): the plan, the rows between the
// products [S, ld_h], their codes and scales, the experts' rows [S, ld_y].
struct ExpertsPlan {
    int64_t S, F_pad, ld_h, ld_y;
    size_t off_offsets, off_rows, off_counts, off_h, off_q, off_scale, off_y, bytes;
};

ExpertsPlan plan_experts_layer(int64_t T, int64_t top_k, int64_t E, int64_t F, int64_t N, cr_dtype dt)
{
    ExpertsPlan p{};
    const int64_t es = elem_size(dt), row = 16 / es;
    p.S = T * top_k;
    p.F_pad = pad256(F);
    p.ld_h = (F + row - 1) / row * row;
    p.ld_y = (N + row - 1) / row * row;
    size_t at = 0;
    auto region = [&](size_t bytes) { const size_t o = at; at += up256(bytes); return o; };
    p.off_offsets = region((size_t)(E + 1) * 4);
    p.off_rows = region((size_t)p.S * 4);
    p.off_counts = region(plan_bytes(p.S, E));
    p.off_h = region((size_t)p.S * (size_t)p.ld_h * (size_t)es);
    p.off_q = region((size_t)p.S * (size_t)p.F_pad);
    p.off_scale = region((size_t)p.S * 4);
    p.off_y = region((size_t)p.S * (size_t)p.ld_y * (size_t)es);
    p.bytes = at;
    return p;
}

}  // namespace

extern "C" {

int cr_abi_version(void) { return CR_ABI_VERSION; }

const char *cr_status_string(cr_status s)
{
    switch (s) {
    case CR_OK: return "CR_OK";
    case CR_ERR_INVALID_ARG: return "CR_ERR_INVALID_ARG";
    case CR_ERR_UNSUPPORTED_DTYPE: return "CR_ERR_UNSUPPORTED_DTYPE";
    case CR_ERR_MISALIGNED: return "CR_ERR_MISALIGNED";
    case CR_ERR_TOO_LARGE: return "CR_ERR_TOO_LARGE";
    case CR_ERR_NO_DEVICE: return "CR_ERR_NO_DEVICE";
    case CR_ERR_LAUNCH: return "CR_ERR_LAUNCH";
    default: return "CR_ERR_UNKNOWN";
    }
}

int64_t cr_padded_k(int64_t k) { return k < 1 ? 0 : pad256(k); }

cr_status cr_prep_weight_nvfp4(const uint8_t *w_fp4, int64_t ld_fp4, const uint8_t *w_sf, int64_t ld_sf,
                               const float *global_scale, int64_t n_rows, int64_t K,
                               int8_t *w_s8, int64_t ld_s8, float *w_scale,
                               uint32_t flags, hipStream_t stream)
{
    cr_status s = check_weight(w_fp4, ld_fp4, w_sf, ld_sf, global_scale, n_rows, K, w_s8, ld_s8, w_scale, flags);
    if (s != CR_OK || n_rows == 0) return s;
    if ((s = current_device_ok()) != CR_OK) return s;
    return from_hip(convrot::launch_prep_weight(w_fp4, ld_fp4, w_sf, ld_sf, global_scale, n_rows, K, w_s8,
                                                ld_s8, w_scale, (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream));
}

cr_status cr_quant_act_ex(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu, int64_t M, int64_t K,
                          const float *pre_scale, int8_t *x_s8, int64_t ld_s8, float *x_scale,
                          uint32_t flags, hipStream_t stream)
{
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    cr_status s = check_act(x, x_dtype, ld_x, M, K, swiglu ? 2 * K : K, x_s8, ld_s8, x_scale, flags);
    if (s != CR_OK) return s;
    if (pre_scale && !aligned(pre_scale, 4)) return CR_ERR_MISALIGNED;
    if (M == 0) return CR_OK;
    if ((s = current_device_ok()) != CR_OK) return s;
    const bool tp = (flags & CR_FLAG_FORCE_TWO_PASS) != 0;
    const bool tr = (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0;
    return from_hip(swiglu
        ? convrot::launch_quant_act_swiglu(x, (int)x_dtype, ld_x, M, K, pre_scale, x_s8, ld_s8, x_scale, tp, tr, stream)
        : convrot::launch_quant_act(x, (int)x_dtype, ld_x, M, K, pre_scale, x_s8, ld_s8, x_scale, tp, tr, stream));
}

cr_status cr_quant_act(const void *x, cr_dtype x_dtype, int64_t ld_x, int64_t M, int64_t K,
                       int8_t *x_s8, int64_t ld_s8, float *x_scale, uint32_t flags, hipStream_t stream)
{
    return cr_quant_act_ex(x, x_dtype, ld_x, 0, M, K, nullptr, x_s8, ld_s8, x_scale, flags, stream);
}

cr_status cr_quant_act_swiglu(const void *h, cr_dtype h_dtype, int64_t ld_h, int64_t M, int64_t F,
                              int8_t *x_s8, int64_t ld_s8, float *x_scale, uint32_t flags, hipStream_t stream)
{
    return cr_quant_act_ex(h, h_dtype, ld_h, 1, M, F, nullptr, x_s8, ld_s8, x_scale, flags, stream);
}

cr_status cr_quant_act_rmsnorm(const void *x, cr_dtype x_dtype, int64_t ld_x, const void *residual, int64_t ld_res,
                               void *sum, int64_t ld_sum, const float *weight, float eps, int64_t M, int64_t K,
                               int8_t *x_s8, int64_t ld_s8, float *x_scale, uint32_t flags, hipStream_t stream)
{
    cr_status s = check_act(x, x_dtype, ld_x, M, K, K, x_s8, ld_s8, x_scale, flags);
    if (s != CR_OK) return s;
    if (!(eps >= 0.0f) || eps > 3.402823466e38f) return CR_ERR_INVALID_ARG;
    if (sum && !residual) return CR_ERR_INVALID_ARG;
    if ((residual && ld_res < K) || (sum && ld_sum < K)) return CR_ERR_INVALID_ARG;
    const int64_t es = elem_size(x_dtype);
    if (residual && (!aligned(residual, 16) || (ld_res * es) % 16 != 0)) return CR_ERR_MISALIGNED;
    if (sum && (!aligned(sum, 16) || (ld_sum * es) % 16 != 0)) return CR_ERR_MISALIGNED;
    if ((sum && sum == x && ld_sum != ld_x) || (sum && sum == residual && ld_sum != ld_res)) return CR_ERR_INVALID_ARG;
    if (weight && !aligned(weight, 4)) return CR_ERR_MISALIGNED;
    if (M == 0) return CR_OK;
    if ((s = current_device_ok()) != CR_OK) return s;
    return from_hip(convrot::launch_quant_act_rmsnorm(x, (int)x_dtype, ld_x, residual, ld_res, sum, ld_sum, weight,
                                                      eps, M, K, x_s8, ld_s8, x_scale,
                                                      (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                      (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, current_cus(), stream));
}

cr_status cr_swiglu(const void *h, cr_dtype h_dtype, int64_t ld_h, int64_t M, int64_t F,
                    float *out, int64_t ld_out, hipStream_t stream)
{
    if (M > 0 && (!h || !out)) return CR_ERR_INVALID_ARG;
    if (h_dtype != CR_BF16 && h_dtype != CR_FP16 && h_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || F < 1 || F > ((int64_t)1 << 40) || M > ((int64_t)1 << 40) / F) return CR_ERR_INVALID_ARG;
    if (ld_h < 2 * F || ld_out < F) return CR_ERR_INVALID_ARG;
    if (!aligned(h, (size_t)elem_size(h_dtype)) || !aligned(out, 4)) return CR_ERR_MISALIGNED;
    if (M == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_swiglu(h, (int)h_dtype, ld_h, M, F, out, ld_out, stream));
}

cr_status cr_gemm_s8_rowscale_bias(const int8_t *a_s8, int64_t lda, const float *a_scale,
                                   const int8_t *b_s8, int64_t ldb, const float *b_scale,
                                   const float *bias, int64_t M, int64_t N, int64_t K_pad,
                                   void *c, cr_dtype c_dtype, int64_t ldc, hipStream_t stream)
{
    cr_status s = check_gemm(a_s8, lda, a_scale, b_s8, ldb, b_scale, M, N, K_pad, c, c_dtype, ldc);
    if (s != CR_OK) return s;
    if (bias && c_dtype == CR_I32) return CR_ERR_INVALID_ARG;
    if (bias && !aligned(bias, 4)) return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;
    if ((s = current_device_ok()) != CR_OK) return s;
    return from_hip(convrot::launch_gemm_s8(a_s8, lda, a_scale, b_s8, ldb, b_scale, bias, M, N, K_pad, c,
                                            (int)c_dtype, ldc, stream));
}

cr_status cr_gemm_s8_rowscale(const int8_t *a_s8, int64_t lda, const float *a_scale,
                              const int8_t *b_s8, int64_t ldb, const float *b_scale,
                              int64_t M, int64_t N, int64_t K_pad,
                              void *c, cr_dtype c_dtype, int64_t ldc, hipStream_t stream)
{
    return cr_gemm_s8_rowscale_bias(a_s8, lda, a_scale, b_s8, ldb, b_scale, nullptr, M, N, K_pad, c,
                                    c_dtype, ldc, stream);
}

cr_status cr_weight_amax_nvfp4(const uint8_t *w_fp4, int64_t ld_fp4, const uint8_t *w_sf, int64_t ld_sf,
                               const float *global_scale, int64_t n_rows, int64_t K, float *w_amax,
                               uint32_t flags, hipStream_t stream)
{
    if (n_rows > 0 && (!w_fp4 || !w_sf || !global_scale || !w_amax)) return CR_ERR_INVALID_ARG;
    if (n_rows < 0 || K < 1 || n_rows > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    if (pad256(K) > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_fp4 < (K + 1) / 2 || ld_sf < (K + 15) / 16) return CR_ERR_INVALID_ARG;
    if (!aligned(w_fp4, 16) || ld_fp4 % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(global_scale, 4) || !aligned(w_amax, 4)) return CR_ERR_MISALIGNED;
    if (n_rows == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_weight_amax(w_fp4, ld_fp4, w_sf, ld_sf, global_scale, n_rows, K, w_amax,
                                                (flags & CR_FLAG_FORCE_TWO_PASS) != 0, stream));
}

cr_status cr_gemm_nvfp4_fused(const int8_t *a_s8, int64_t lda, const float *a_scale,
                              const uint8_t *w_fp4, int64_t ld_fp4, const uint8_t *w_sf, int64_t ld_sf,
                              const float *global_scale, const float *w_amax, const float *bias,
                              int64_t M, int64_t N, int64_t K, void *c, cr_dtype c_dtype, int64_t ldc,
                              uint32_t flags, hipStream_t stream)
{
    cr_status s0 = check_fused(a_s8, lda, a_scale, w_fp4, ld_fp4, w_sf, ld_sf, global_scale, w_amax, bias, M, N, K,
                               c, c_dtype, ldc, flags);
    if (s0 != CR_OK || M == 0 || N == 0) return s0;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_gemm_nvfp4_fused(a_s8, lda, a_scale, w_fp4, ld_fp4, w_sf, ld_sf, global_scale,
                                                     w_amax, bias, M, N, K, c, (int)c_dtype, ldc,
                                                     (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream));
}

cr_status cr_linear_nvfp4_plan(int64_t M, int64_t N, int64_t K, size_t max_tile_bytes,
                               int64_t *rows_per_chunk, int64_t *nchunks)
{
    if (!rows_per_chunk || !nchunks) return CR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K < 1) return CR_ERR_INVALID_ARG;
    if (pad256(K) > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    const LayerPlan p = plan_layer(M, N, K, max_tile_bytes);
    *rows_per_chunk = p.R;
    *nchunks = p.nchunks;
    return CR_OK;
}

size_t cr_linear_nvfp4_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t max_tile_bytes)
{
    if (M < 1 || N < 1 || K < 1 || pad256(K) > CR_MAX_K_PAD) return 0;   // an empty layer needs none
    return plan_layer(M, N, K, max_tile_bytes).bytes;
}

cr_status cr_linear_nvfp4_ex(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu,
                             int64_t M, int64_t K, const float *pre_scale,
                             const uint8_t *w_fp4, int64_t ld_fp4,
                             const uint8_t *w_sf, int64_t ld_sf, const float *global_scale,
                             int64_t N, const float *bias, void *out, cr_dtype out_dtype, int64_t ldc,
                             void *workspace, size_t ws_bytes, size_t max_tile_bytes,
                             uint32_t flags, hipStream_t s_main, hipStream_t s_aux)
{
    if (out_dtype == CR_I32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 1) return CR_ERR_INVALID_ARG;
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    if (pad256(K) > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (M == 0 || N == 0) {
        // an empty layer: the arguments that do not depend on the empty extent are checked
        // as for any other call, and nothing is enqueued
        if (x_dtype != CR_BF16 && x_dtype != CR_FP16 && x_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
        if (out_dtype != CR_BF16 && out_dtype != CR_FP16 && out_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
        if (check_flags(flags) != CR_OK || ld_x < (swiglu ? 2 * K : K) || ldc < N) return CR_ERR_INVALID_ARG;
        if ((M > 0 && !x) || (N > 0 && (!w_fp4 || !w_sf || !global_scale))) return CR_ERR_INVALID_ARG;
        if (ld_fp4 < (K + 1) / 2 || ld_sf < (K + 15) / 16) return CR_ERR_INVALID_ARG;
        if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
        if (!aligned(w_fp4, 16) || ld_fp4 % 16 != 0) return CR_ERR_MISALIGNED;
        return CR_OK;
    }
    if (!workspace || !out) return CR_ERR_INVALID_ARG;
    const LayerPlan p = plan_layer(M, N, K, max_tile_bytes);
    if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
    if (ws_bytes < p.bytes) return CR_ERR_TOO_LARGE;
    int8_t *ws = static_cast<int8_t *>(workspace);
    int8_t *x_s8 = ws;
    float *x_scale = reinterpret_cast<float *>(ws + p.off_xscale);
    if (p.fused) {
        cr_status s = check_act(x, x_dtype, ld_x, M, K, swiglu ? 2 * K : K, x_s8, p.K_pad, x_scale, flags);
        if (s != CR_OK) return s;
        s = check_fused(x_s8, p.K_pad, x_scale, w_fp4, ld_fp4, w_sf, ld_sf, global_scale, nullptr, bias, M, N, K,
                        out, out_dtype, ldc, flags);
        if (s != CR_OK) return s;
        if (pre_scale && !aligned(pre_scale, 4)) return CR_ERR_MISALIGNED;
        if ((s = current_device_ok()) != CR_OK) return s;
        const bool tp = (flags & CR_FLAG_FORCE_TWO_PASS) != 0;
        // both launches on s_main: they are short, kernels running side by side on this
        // chip take as long as one after the other, and cross-stream waits would cost more
        // than the whole activation preparation
        hipError_t e = swiglu
            ? convrot::launch_quant_act_swiglu(x, (int)x_dtype, ld_x, M, K, pre_scale, x_s8, p.K_pad, x_scale, tp, true, s_main)
            : convrot::launch_quant_act(x, (int)x_dtype, ld_x, M, K, pre_scale, x_s8, p.K_pad, x_scale, tp, true, s_main);
        if (e != hipSuccess) return CR_ERR_LAUNCH;
        return from_hip(convrot::launch_gemm_nvfp4_fused(x_s8, p.K_pad, x_scale, w_fp4, ld_fp4, w_sf, ld_sf,
                                                         global_scale, nullptr, bias, M, N, K, out, (int)out_dtype,
                                                         ldc, true, s_main));
    }
    int8_t *tile[2] = {ws + p.off_tile[0], ws + p.off_tile[1]};
    float *tscale[2] = {reinterpret_cast<float *>(ws + p.off_tscale[0]),
                        reinterpret_cast<float *>(ws + p.off_tscale[1])};
    // validate every call of the plan before enqueueing anything
    cr_status s = check_act(x, x_dtype, ld_x, M, K, swiglu ? 2 * K : K, x_s8, p.K_pad, x_scale, flags);
    if (s != CR_OK) return s;
    s = check_weight(w_fp4, ld_fp4, w_sf, ld_sf, global_scale, p.R < N ? p.R : N, K, tile[0], p.K_pad,
                     tscale[0], flags);
    if (s != CR_OK) return s;
    s = check_gemm(x_s8, p.K_pad, x_scale, tile[0], p.K_pad, tscale[0], M, p.R < N ? p.R : N, p.K_pad,
                   out, out_dtype, ldc);
    if (s != CR_OK) return s;
    if ((pre_scale && !aligned(pre_scale, 4)) || (bias && !aligned(bias, 4))) return CR_ERR_MISALIGNED;
    if ((s = current_device_ok()) != CR_OK) return s;

    const bool tp = (flags & CR_FLAG_FORCE_TWO_PASS) != 0;
    const int64_t es = elem_size(out_dtype);
    // with a second stream and several chunks, chunk c+1 is prepared while chunk c
    // multiplies (and the first while the activation is prepared), the overlap a caller asks
    // for by passing s_aux.  On this chip it measured 1 % (two chunks) to 3.5 % (seven
    // chunks) slower than staging every chunk on s_main: a preparation kernel started beside
    // a running GEMM waits for the compute units the GEMM holds and delays the next GEMM's
    // workgroups.  A single chunk has only the activation preparation to run beside, which
    // gains nothing either, while the two cross-stream waits cost about as much as a small
    // layer's activation preparation.
    const bool overlap = s_aux != nullptr && s_aux != s_main && p.nchunks > 1;
    PooledEvents evs(overlap);
    if (overlap && !evs.ok()) return CR_ERR_LAUNCH;
    hipEvent_t ev_start = nullptr, ev_prep[2] = {nullptr, nullptr}, ev_gemm[2] = {nullptr, nullptr};
    if (overlap) {
        ev_start = evs[0];
        ev_prep[0] = evs[1]; ev_prep[1] = evs[2];
        ev_gemm[0] = evs[3]; ev_gemm[1] = evs[4];
    }

    if (overlap) {
        // the staging stream must not run ahead of work already queued on s_main
        if (hipEventRecord(ev_start, s_main) != hipSuccess) return CR_ERR_LAUNCH;
        if (hipStreamWaitEvent(s_aux, ev_start, 0) != hipSuccess) return CR_ERR_LAUNCH;
    }
    // both S8 operands live only in the workspace: they use the block-transposed column
    // order, which skips one LDS transposition per block and leaves every int32 sum as is
    hipError_t e = swiglu
        ? convrot::launch_quant_act_swiglu(x, (int)x_dtype, ld_x, M, K, pre_scale, x_s8, p.K_pad, x_scale, tp, true, s_main)
        : convrot::launch_quant_act(x, (int)x_dtype, ld_x, M, K, pre_scale, x_s8, p.K_pad, x_scale, tp, true, s_main);
    if (e != hipSuccess) return CR_ERR_LAUNCH;

    for (int64_t c = 0; c < p.nchunks; c++) {
        const int b = (int)(c & 1);
        const int64_t n0 = c * p.R;
        const int64_t rows = (N - n0) < p.R ? (N - n0) : p.R;
        hipStream_t sp = overlap ? s_aux : s_main;
        if (overlap && c >= 2 && hipStreamWaitEvent(s_aux, ev_gemm[b], 0) != hipSuccess) return CR_ERR_LAUNCH;
        e = convrot::launch_prep_weight(w_fp4 + n0 * ld_fp4, ld_fp4, w_sf + n0 * ld_sf, ld_sf, global_scale,
                                        rows, K, tile[b], p.K_pad, tscale[b], tp, true, sp);
        if (e != hipSuccess) return CR_ERR_LAUNCH;
        if (overlap) {
            if (hipEventRecord(ev_prep[b], s_aux) != hipSuccess) return CR_ERR_LAUNCH;
            if (hipStreamWaitEvent(s_main, ev_prep[b], 0) != hipSuccess) return CR_ERR_LAUNCH;
        }
        e = convrot::launch_gemm_s8(x_s8, p.K_pad, x_scale, tile[b], p.K_pad, tscale[b],
                                    bias ? bias + n0 : nullptr, M, rows, p.K_pad,
                                    static_cast<int8_t *>(out) + n0 * es, (int)out_dtype, ldc, s_main);
        if (e != hipSuccess) return CR_ERR_LAUNCH;
        if (overlap && hipEventRecord(ev_gemm[b], s_main) != hipSuccess) return CR_ERR_LAUNCH;
    }
    return CR_OK;
}

cr_status cr_linear_nvfp4(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu,
                          int64_t M, int64_t K,
                          const uint8_t *w_fp4, int64_t ld_fp4,
                          const uint8_t *w_sf, int64_t ld_sf, const float *global_scale,
                          int64_t N, void *out, cr_dtype out_dtype, int64_t ldc,
                          void *workspace, size_t ws_bytes, size_t max_tile_bytes,
                          uint32_t flags, hipStream_t s_main, hipStream_t s_aux)
{
    return cr_linear_nvfp4_ex(x, x_dtype, ld_x, swiglu, M, K, nullptr, w_fp4, ld_fp4, w_sf, ld_sf,
                              global_scale, N, nullptr, out, out_dtype, ldc, workspace, ws_bytes,
                              max_tile_bytes, flags, s_main, s_aux);
}

cr_status cr_quant_weight_w4(const void *w, cr_dtype w_dtype, int64_t ld_w, int64_t N, int64_t K,
                             uint8_t *w_s4, int64_t ld_s4, float *w_scale, uint32_t flags, hipStream_t stream)
{
    if (N > 0 && (!w || !w_s4 || !w_scale)) return CR_ERR_INVALID_ARG;
    if (w_dtype != CR_BF16 && w_dtype != CR_FP16 && w_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (N < 0 || K < 1 || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_w < K || ld_s4 < kp / 2) return CR_ERR_INVALID_ARG;
    if (!aligned(w, 16) || (ld_w * elem_size(w_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(w_s4, 16) || ld_s4 % 16 != 0 || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
    if (N == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_quant_weight_w4(w, (int)w_dtype, ld_w, N, K, w_s4, ld_s4, w_scale,
                                                    (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                    (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream));
}

cr_status cr_gemm_s8s4_rowscale(const int8_t *a_s8, int64_t lda, const float *a_scale,
                                const uint8_t *b_s4, int64_t ldb, const float *b_scale, const float *bias,
                                int64_t M, int64_t N, int64_t K_pad, void *c, cr_dtype c_dtype, int64_t ldc,
                                hipStream_t stream)
{
    if ((M > 0 && !a_s8) || (N > 0 && !b_s4) || (M > 0 && N > 0 && !c)) return CR_ERR_INVALID_ARG;
    if (c_dtype != CR_BF16 && c_dtype != CR_FP16 && c_dtype != CR_FP32 && c_dtype != CR_I32)
        return CR_ERR_UNSUPPORTED_DTYPE;
    if (c_dtype != CR_I32 && ((M > 0 && !a_scale) || (N > 0 && !b_scale))) return CR_ERR_INVALID_ARG;
    if (bias && c_dtype == CR_I32) return CR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K_pad < 1 || K_pad % 256 != 0 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (K_pad > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (lda < K_pad || ldb < K_pad / 2 || ldc < N) return CR_ERR_INVALID_ARG;   // ldb in bytes
    if (!aligned(a_s8, 16) || !aligned(b_s4, 16) || lda % 16 != 0 || ldb % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(c, (size_t)elem_size(c_dtype))) return CR_ERR_MISALIGNED;
    if ((a_scale && !aligned(a_scale, 4)) || (b_scale && !aligned(b_scale, 4)) || (bias && !aligned(bias, 4)))
        return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_gemm_s8s4(a_s8, lda, a_scale, b_s4, ldb, b_scale, bias, M, N, K_pad, c,
                                              (int)c_dtype, ldc, stream));
}

size_t cr_linear_w4a8_workspace_bytes(int64_t M, int64_t K)
{
    if (M < 1 || K < 1 || pad256(K) > CR_MAX_K_PAD) return 0;
    return up256(up256((size_t)M * (size_t)pad256(K)) + (size_t)M * 4);
}

cr_status cr_linear_w4a8(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu, int64_t M, int64_t K,
                         const uint8_t *w_s4, int64_t ld_s4, const float *w_scale, int64_t N, const float *bias,
                         void *out, cr_dtype out_dtype, int64_t ldc, void *workspace, size_t ws_bytes,
                         uint32_t flags, hipStream_t stream)
{
    if (x_dtype != CR_BF16 && x_dtype != CR_FP16 && x_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (out_dtype != CR_BF16 && out_dtype != CR_FP16 && out_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 1 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (ld_x < (swiglu ? 2 * K : K) || ld_s4 < kp / 2 || ldc < N) return CR_ERR_INVALID_ARG;
    if ((M > 0 && !x) || (N > 0 && (!w_s4 || !w_scale)) || (M > 0 && N > 0 && !out)) return CR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(w_s4, 16) || ld_s4 % 16 != 0 || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
    if ((bias && !aligned(bias, 4)) || !aligned(out, (size_t)elem_size(out_dtype))) return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;       // an empty layer: nothing to enqueue, no workspace
    if (!workspace) return CR_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
    if (ws_bytes < cr_linear_w4a8_workspace_bytes(M, K)) return CR_ERR_TOO_LARGE;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    int8_t *x_s8 = static_cast<int8_t *>(workspace);
    float *x_scale = reinterpret_cast<float *>(x_s8 + up256((size_t)M * (size_t)kp));
    const bool tp = (flags & CR_FLAG_FORCE_TWO_PASS) != 0;
    const bool tr = (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0;
    hipError_t e = swiglu
        ? convrot::launch_quant_act_swiglu(x, (int)x_dtype, ld_x, M, K, nullptr, x_s8, kp, x_scale, tp, tr, stream)
        : convrot::launch_quant_act(x, (int)x_dtype, ld_x, M, K, nullptr, x_s8, kp, x_scale, tp, tr, stream);
    if (e != hipSuccess) return CR_ERR_LAUNCH;
    return from_hip(convrot::launch_gemm_s8s4(x_s8, kp, x_scale, w_s4, ld_s4, w_scale, bias, M, N, kp, out,
                                              (int)out_dtype, ldc, stream));
}

cr_status cr_quant_act_w4(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu, int64_t M, int64_t K,
                          uint8_t *x_s4, int64_t ld_s4, float *x_scale, uint32_t flags, hipStream_t stream)
{
    if (M > 0 && (!x || !x_s4 || !x_scale)) return CR_ERR_INVALID_ARG;
    if (x_dtype != CR_BF16 && x_dtype != CR_FP16 && x_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || K < 1 || M > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_x < (swiglu ? 2 * K : K) || ld_s4 < kp / 2) return CR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(x_s4, 16) || ld_s4 % 16 != 0 || !aligned(x_scale, 4)) return CR_ERR_MISALIGNED;
    if (M == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_quant_act_w4(x, (int)x_dtype, ld_x, swiglu != 0, M, K, x_s4, ld_s4, x_scale,
                                                 (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                 (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream));
}

cr_status cr_gemm_s4s4_rowscale(const uint8_t *a_s4, int64_t lda, const float *a_scale,
                                const uint8_t *b_s4, int64_t ldb, const float *b_scale, const float *bias,
                                int64_t M, int64_t N, int64_t K_pad, void *c, cr_dtype c_dtype, int64_t ldc,
                                hipStream_t stream)
{
    if ((M > 0 && !a_s4) || (N > 0 && !b_s4) || (M > 0 && N > 0 && !c)) return CR_ERR_INVALID_ARG;
    if (c_dtype != CR_BF16 && c_dtype != CR_FP16 && c_dtype != CR_FP32 && c_dtype != CR_I32)
        return CR_ERR_UNSUPPORTED_DTYPE;
    if (c_dtype != CR_I32 && ((M > 0 && !a_scale) || (N > 0 && !b_scale))) return CR_ERR_INVALID_ARG;
    if (bias && c_dtype == CR_I32) return CR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K_pad < 1 || K_pad % 256 != 0 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (K_pad > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (lda < K_pad / 2 || ldb < K_pad / 2 || ldc < N) return CR_ERR_INVALID_ARG;   // lda, ldb in bytes
    if (!aligned(a_s4, 16) || !aligned(b_s4, 16) || lda % 16 != 0 || ldb % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(c, (size_t)elem_size(c_dtype))) return CR_ERR_MISALIGNED;
    if ((a_scale && !aligned(a_scale, 4)) || (b_scale && !aligned(b_scale, 4)) || (bias && !aligned(bias, 4)))
        return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_gemm_s4s4(a_s4, lda, a_scale, b_s4, ldb, b_scale, bias, M, N, K_pad, c,
                                              (int)c_dtype, ldc, stream));
}

size_t cr_linear_w4a4_workspace_bytes(int64_t M, int64_t K)
{
    if (M < 1 || K < 1 || pad256(K) > CR_MAX_K_PAD) return 0;
    return up256(up256((size_t)M * (size_t)(pad256(K) / 2)) + (size_t)M * 4);
}

cr_status cr_linear_w4a4(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu, int64_t M, int64_t K,
                         const uint8_t *w_s4, int64_t ld_s4, const float *w_scale, int64_t N, const float *bias,
                         void *out, cr_dtype out_dtype, int64_t ldc, void *workspace, size_t ws_bytes,
                         uint32_t flags, hipStream_t stream)
{
    if (x_dtype != CR_BF16 && x_dtype != CR_FP16 && x_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (out_dtype != CR_BF16 && out_dtype != CR_FP16 && out_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 1 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (ld_x < (swiglu ? 2 * K : K) || ld_s4 < kp / 2 || ldc < N) return CR_ERR_INVALID_ARG;
    if ((M > 0 && !x) || (N > 0 && (!w_s4 || !w_scale)) || (M > 0 && N > 0 && !out)) return CR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(w_s4, 16) || ld_s4 % 16 != 0 || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
    if ((bias && !aligned(bias, 4)) || !aligned(out, (size_t)elem_size(out_dtype))) return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;       // an empty layer: nothing to enqueue, no workspace
    if (!workspace) return CR_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
    if (ws_bytes < cr_linear_w4a4_workspace_bytes(M, K)) return CR_ERR_TOO_LARGE;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    uint8_t *x_s4 = static_cast<uint8_t *>(workspace);
    float *x_scale = reinterpret_cast<float *>(x_s4 + up256((size_t)M * (size_t)(kp / 2)));
    hipError_t e = convrot::launch_quant_act_w4(x, (int)x_dtype, ld_x, swiglu != 0, M, K, x_s4, kp / 2, x_scale,
                                                (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream);
    if (e != hipSuccess) return CR_ERR_LAUNCH;
    return from_hip(convrot::launch_gemm_s4s4(x_s4, kp / 2, x_scale, w_s4, ld_s4, w_scale, bias, M, N, kp, out,
                                              (int)out_dtype, ldc, stream));
}

cr_status cr_quant_weight_w4_e2m3(const void *w, cr_dtype w_dtype, int64_t ld_w, int64_t N, int64_t K,
                                  uint8_t *w_f6, int64_t ld_f6, float *w_scale, uint32_t flags, hipStream_t stream)
{
    if (N > 0 && (!w || !w_f6 || !w_scale)) return CR_ERR_INVALID_ARG;
    if (w_dtype != CR_BF16 && w_dtype != CR_FP16 && w_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (N < 0 || K < 1 || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_w < K || ld_f6 < 3 * kp) return CR_ERR_INVALID_ARG;
    if (!aligned(w, 16) || (ld_w * elem_size(w_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(w_f6, 16) || ld_f6 % 16 != 0 || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
    if (N == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_quant_weight_e2m3(w, (int)w_dtype, ld_w, N, K, w_f6, ld_f6, w_scale,
                                                      (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                      (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream));
}

cr_status cr_repack_w4_e2m3(const uint8_t *w_s4, int64_t ld_s4, int64_t N, int64_t K_pad, uint8_t *w_f6,
                            int64_t ld_f6, hipStream_t stream)
{
    if (N > 0 && (!w_s4 || !w_f6)) return CR_ERR_INVALID_ARG;
    if (N < 0 || N > kMaxRows || K_pad < 1 || K_pad % 256 != 0) return CR_ERR_INVALID_ARG;
    if (K_pad > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_s4 < K_pad / 2 || ld_f6 < 3 * K_pad) return CR_ERR_INVALID_ARG;
    if (!aligned(w_s4, 16) || ld_s4 % 16 != 0 || !aligned(w_f6, 16) || ld_f6 % 16 != 0) return CR_ERR_MISALIGNED;
    if (N == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_repack_w4_e2m3(w_s4, ld_s4, N, K_pad, w_f6, ld_f6, stream));
}

cr_status cr_quant_act_w4_e2m3(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu, int64_t M, int64_t K,
                               uint8_t *x_f6, int64_t ld_f6, float *x_scale, uint32_t flags, hipStream_t stream)
{
    if (M > 0 && (!x || !x_f6 || !x_scale)) return CR_ERR_INVALID_ARG;
    if (x_dtype != CR_BF16 && x_dtype != CR_FP16 && x_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || K < 1 || M > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (ld_x < (swiglu ? 2 * K : K) || ld_f6 < 3 * kp) return CR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(x_f6, 16) || ld_f6 % 16 != 0 || !aligned(x_scale, 4)) return CR_ERR_MISALIGNED;
    if (M == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_quant_act_e2m3(x, (int)x_dtype, ld_x, swiglu != 0, M, K, x_f6, ld_f6, x_scale,
                                                   (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                   (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream));
}

cr_status cr_gemm_e2m3_rowscale(const uint8_t *a_f6, int64_t lda, const float *a_scale,
                                const uint8_t *b_f6, int64_t ldb, const float *b_scale, const float *bias,
                                int64_t M, int64_t N, int64_t K_pad, void *c, cr_dtype c_dtype, int64_t ldc,
                                hipStream_t stream)
{
    if ((M > 0 && !a_f6) || (N > 0 && !b_f6) || (M > 0 && N > 0 && !c)) return CR_ERR_INVALID_ARG;
    if (c_dtype != CR_BF16 && c_dtype != CR_FP16 && c_dtype != CR_FP32 && c_dtype != CR_I32)
        return CR_ERR_UNSUPPORTED_DTYPE;
    if (c_dtype != CR_I32 && ((M > 0 && !a_scale) || (N > 0 && !b_scale))) return CR_ERR_INVALID_ARG;
    if (bias && c_dtype == CR_I32) return CR_ERR_INVALID_ARG;
    if (M < 0 || N < 0 || K_pad < 1 || K_pad % 256 != 0 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (K_pad > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (lda < 3 * K_pad || ldb < 3 * K_pad || ldc < N) return CR_ERR_INVALID_ARG;   // bytes per quad of rows
    if (!aligned(a_f6, 16) || !aligned(b_f6, 16) || lda % 16 != 0 || ldb % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(c, (size_t)elem_size(c_dtype))) return CR_ERR_MISALIGNED;
    if ((a_scale && !aligned(a_scale, 4)) || (b_scale && !aligned(b_scale, 4)) || (bias && !aligned(bias, 4)))
        return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    return from_hip(convrot::launch_gemm_e2m3(a_f6, lda, a_scale, b_f6, ldb, b_scale, bias, M, N, K_pad, c,
                                              (int)c_dtype, ldc, stream));
}

size_t cr_linear_w4a4_e2m3_workspace_bytes(int64_t M, int64_t K)
{
    if (M < 1 || K < 1 || pad256(K) > CR_MAX_K_PAD) return 0;
    return up256(up256((size_t)((M + 3) / 4) * (size_t)(3 * pad256(K))) + (size_t)M * 4);
}

cr_status cr_linear_w4a4_e2m3(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu, int64_t M, int64_t K,
                              const uint8_t *w_f6, int64_t ld_f6, const float *w_scale, int64_t N,
                              const float *bias, void *out, cr_dtype out_dtype, int64_t ldc, void *workspace,
                              size_t ws_bytes, uint32_t flags, hipStream_t stream)
{
    if (x_dtype != CR_BF16 && x_dtype != CR_FP16 && x_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (out_dtype != CR_BF16 && out_dtype != CR_FP16 && out_dtype != CR_FP32) return CR_ERR_UNSUPPORTED_DTYPE;
    if (M < 0 || N < 0 || K < 1 || M > kMaxRows || N > kMaxRows) return CR_ERR_INVALID_ARG;
    if (check_flags(flags) != CR_OK) return CR_ERR_INVALID_ARG;
    if (swiglu && K > (int64_t)1 << 40) return CR_ERR_TOO_LARGE;
    const int64_t kp = pad256(K);
    if (kp > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (((M + 255) / 256) * ((N + 255) / 256) > (int64_t)(UINT32_MAX / 512)) return CR_ERR_TOO_LARGE;
    if (ld_x < (swiglu ? 2 * K : K) || ld_f6 < 3 * kp || ldc < N) return CR_ERR_INVALID_ARG;
    if ((M > 0 && !x) || (N > 0 && (!w_f6 || !w_scale)) || (M > 0 && N > 0 && !out)) return CR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || (ld_x * elem_size(x_dtype)) % 16 != 0) return CR_ERR_MISALIGNED;
    if (!aligned(w_f6, 16) || ld_f6 % 16 != 0 || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
    if ((bias && !aligned(bias, 4)) || !aligned(out, (size_t)elem_size(out_dtype))) return CR_ERR_MISALIGNED;
    if (M == 0 || N == 0) return CR_OK;       // an empty layer: nothing to enqueue, no workspace
    if (!workspace) return CR_ERR_INVALID_ARG;
    if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
    if (ws_bytes < cr_linear_w4a4_e2m3_workspace_bytes(M, K)) return CR_ERR_TOO_LARGE;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    const int64_t lf = 3 * kp;                  // one quad of rows
    uint8_t *x_f6 = static_cast<uint8_t *>(workspace);
    float *x_scale = reinterpret_cast<float *>(x_f6 + up256((size_t)((M + 3) / 4) * (size_t)lf));
    hipError_t e = convrot::launch_quant_act_e2m3(x, (int)x_dtype, ld_x, swiglu != 0, M, K, x_f6, lf, x_scale,
                                                  (flags & CR_FLAG_FORCE_TWO_PASS) != 0,
                                                  (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0, stream);
    if (e != hipSuccess) return CR_ERR_LAUNCH;
    return from_hip(convrot::launch_gemm_e2m3(x_f6, lf, x_scale, w_f6, ld_f6, w_scale, bias, M, N, kp, out,
                                              (int)out_dtype, ldc, stream));
}

cr_status cr_linear_nvfp4_noalloc(const void *x, cr_dtype x_dtype, int64_t ld_x, int swiglu,
                                  int64_t M, int64_t K, const float *pre_scale,
                                  const uint8_t *w_fp4, int64_t ld_fp4,
                                  const uint8_t *w_sf, int64_t ld_sf, const float *global_scale,
                                  int64_t N, const float *bias, void *out, cr_dtype out_dtype, int64_t ldc,
                                  size_t max_tile_bytes, uint32_t flags, hipStream_t stream)
{
    if (M < 0 || N < 0 || K < 1) return CR_ERR_INVALID_ARG;
    if (pad256(K) > CR_MAX_K_PAD) return CR_ERR_TOO_LARGE;
    if (M == 0 || N == 0)    // an empty layer: argument checks only, as in cr_linear_nvfp4_ex
        return cr_linear_nvfp4_ex(x, x_dtype, ld_x, swiglu, M, K, pre_scale, w_fp4, ld_fp4, w_sf, ld_sf,
                                  global_scale, N, bias, out, out_dtype, ldc, nullptr, 0, max_tile_bytes, flags,
                                  stream, nullptr);
    size_t bound = max_tile_bytes;
    if (bound == 0 && M > kFusedMaxRows) {
        bound = noalloc_tile_bound(M, K);
        if (bound == 0) return CR_ERR_TOO_LARGE;
    }
    if (plan_layer(M, N, K, bound).bytes > CR_NOALLOC_SCRATCH_BYTES) return CR_ERR_TOO_LARGE;
    cr_status s = current_device_ok();
    if (s != CR_OK) return s;
    void *ws = nullptr;
    if ((s = scratch_for_current_device(&ws)) != CR_OK) return s;
    // serial staging on `stream`: no second stream, so no events are needed
    return cr_linear_nvfp4_ex(x, x_dtype, ld_x, swiglu, M, K, pre_scale, w_fp4, ld_fp4, w_sf, ld_sf, global_scale,
                              N, bias, out, out_dtype, ldc, ws, CR_NOALLOC_SCRATCH_BYTES, bound, flags, stream,
                              nullptr);
}

cr_status cr_rope_append_kv8(const void *qkv, cr_dtype dtype, int64_t ld_qkv, int64_t T, int64_t B,
                             const int32_t *cu_seqlens, const int32_t *kv_lens, int64_t max_new,
                             int64_t Hq, int64_t Hkv, int64_t D, const float *q_weight, const float *k_weight,
                             float eps, const int32_t *pos, int64_t ld_pos, int64_t n_axes, const double *freq,
                             const int32_t *axis, void *q_out, int64_t ld_q, const cr_kv8_cache *cache,
                             uint32_t flags, hipStream_t stream)
{
    cr_status s = check_kv8(dtype, T, B, cu_seqlens, kv_lens, Hq, Hkv, D, cache, Hkv > 0);
    if (s != CR_OK) return s;
    const bool any = T > 0 && B > 0 && Hq + Hkv > 0;
    if (flags & ~(uint32_t)CR_FLAG_ROPE_INTERLEAVED) return CR_ERR_INVALID_ARG;
    if (max_new < 0 || n_axes < 1 || n_axes > 4 || ld_pos < n_axes) return CR_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || eps > 3.402823466e38f) return CR_ERR_INVALID_ARG;
    if ((s = check_rows16(qkv, ld_qkv, (Hq + 2 * Hkv) * D, any)) != CR_OK) return s;
    if (Hq > 0 && (s = check_rows16(q_out, ld_q, Hq * D, any)) != CR_OK) return s;
    if (q_out && q_out == qkv && Hq > 0 && ld_q != ld_qkv) return CR_ERR_INVALID_ARG;
    if (any && (!pos || !freq || !axis)) return CR_ERR_INVALID_ARG;
    if (!aligned(pos, 4) || !aligned(freq, 8) || !aligned(axis, 4) || !aligned(q_weight, 4) || !aligned(k_weight, 4))
        return CR_ERR_MISALIGNED;
    if (max_new > T) max_new = T;
    if (!any || max_new == 0) return CR_OK;
    // workgroups of at most 512 threads, at most one per page visited and head; a dispatch counts
    // work-items in 32 bits
    const int64_t visits = (max_new + CR_KV8_PAGE - 2) / CR_KV8_PAGE + 1;
    if (B > (int64_t)(UINT32_MAX / 512) / visits / (Hq + Hkv)) return CR_ERR_TOO_LARGE;
    if ((s = current_device_ok()) != CR_OK) return s;
    convrot::RopeLaunch r{};
    r.qkv = qkv; r.dtype = (int)dtype; r.ld_qkv = ld_qkv; r.q_out = q_out; r.ld_q = ld_q;
    r.q_weight = q_weight; r.k_weight = k_weight; r.eps = eps;
    r.pos = pos; r.ld_pos = ld_pos; r.n_axes = (int)n_axes; r.freq = freq; r.axis = axis;
    r.interleaved = (flags & CR_FLAG_ROPE_INTERLEAVED) != 0;
    r.T = T; r.B = B; r.max_new = max_new; r.cu = cu_seqlens; r.kv_lens = kv_lens;
    r.Hq = (int)Hq; r.Hkv = (int)Hkv; r.D = (int)D; r.cache = kv8_ptrs(Hkv > 0 ? cache : nullptr);
    r.cus = current_cus();
    return from_hip(convrot::launch_rope_append_kv8(r, stream));
}

size_t cr_attn_kv8_workspace_bytes(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int64_t Hq, int64_t Hkv,
                                   int64_t D)
{
    convrot::AttnPlan p;
    return attn_plan(T, B, max_q, max_kv, Hq, Hkv, D, &p) ? p.bytes : 0;
}

cr_status cr_attn_kv8(const void *q, cr_dtype dtype, int64_t ld_q, int64_t T, int64_t B,
                      const int32_t *cu_seqlens, const int32_t *kv_lens, int64_t max_q, int64_t max_kv,
                      int64_t Hq, int64_t Hkv, int64_t D, const cr_kv8_cache *cache, float sm_scale,
                      void *out, int64_t ld_out, void *workspace, size_t ws_bytes, uint32_t flags,
                      hipStream_t stream)
{
    cr_status s = check_kv8(dtype, T, B, cu_seqlens, kv_lens, Hq, Hkv, D, cache, true);
    if (s != CR_OK) return s;
    const bool any = T > 0 && B > 0;
    if (flags & ~(uint32_t)CR_FLAG_CAUSAL) return CR_ERR_INVALID_ARG;
    if (!(sm_scale > 0.0f) || sm_scale > 3.402823466e38f) return CR_ERR_INVALID_ARG;
    convrot::AttnPlan p;
    if (!attn_plan(T, B, max_q, max_kv, Hq, Hkv, D, &p)) return CR_ERR_INVALID_ARG;
    if ((s = check_rows16(q, ld_q, Hq * D, any)) != CR_OK) return s;
    if ((s = check_rows16(out, ld_out, Hq * D, any)) != CR_OK) return s;
    if (any && p.bytes > 0) {
        if (!workspace) return CR_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
        if (ws_bytes < p.bytes) return CR_ERR_TOO_LARGE;
    }
    if (!any || max_q == 0) return CR_OK;
    if (p.whole > convrot::kMostBlocks || p.whole + p.tail * p.splits > convrot::kMostBlocks ||
        p.join_groups > convrot::kMostBlocks || T > 4 * convrot::kMostBlocks / Hq)
        return CR_ERR_TOO_LARGE;
    if ((s = current_device_ok()) != CR_OK) return s;
    convrot::AttnLaunch l{};
    l.q = q; l.dtype = (int)dtype; l.ld_q = ld_q; l.out = out; l.ld_out = ld_out; l.T = T; l.B = B;
    l.cu = cu_seqlens; l.kv_lens = kv_lens; l.Hq = (int)Hq; l.Hkv = (int)Hkv; l.D = (int)D;
    l.cache = kv8_ptrs(cache); l.sm_scale = sm_scale; l.causal = (flags & CR_FLAG_CAUSAL) != 0;
    l.workspace = workspace; l.plan = p;
    return from_hip(convrot::launch_attn_kv8(l, stream));
}

cr_status cr_route_experts(const void *logits, cr_dtype dtype, int64_t ld, int64_t T, int64_t E, const float *bias,
                           int64_t n_groups, int64_t top_groups, int64_t group_sum, int64_t top_k, float scale,
                           int32_t *ids, float *weights, uint32_t flags, hipStream_t stream)
{
    if (!is_float(dtype)) return CR_ERR_UNSUPPORTED_DTYPE;
    if (flags & ~(uint32_t)(CR_FLAG_ROUTE_SIGMOID | CR_FLAG_ROUTE_RENORM)) return CR_ERR_INVALID_ARG;
    cr_status s = check_slots(T, top_k, 0, E);
    if (s != CR_OK) return s;
    if (T > 0 && (!logits || !ids || !weights)) return CR_ERR_INVALID_ARG;
    if (ld < E || group_sum < 1 || group_sum > 2) return CR_ERR_INVALID_ARG;
    if (n_groups < 1 || n_groups > CR_MAX_EXPERT_GROUPS || E % n_groups != 0) return CR_ERR_INVALID_ARG;
    if (top_groups < 1 || top_groups > n_groups || top_k > top_groups * (E / n_groups)) return CR_ERR_INVALID_ARG;
    if (!(scale >= -3.402823466e38f && scale <= 3.402823466e38f)) return CR_ERR_INVALID_ARG;
    if (!aligned(logits, (size_t)elem_size(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
        return CR_ERR_MISALIGNED;
    if (T == 0) return CR_OK;
    if (T > convrot::kMostBlocks) return CR_ERR_TOO_LARGE;
    if ((s = current_device_ok()) != CR_OK) return s;
    convrot::RouteLaunch r{};
    r.logits = logits; r.ld = ld; r.T = T; r.E = (int)E; r.G = (int)n_groups; r.top_groups = (int)top_groups;
    r.group_sum = (int)group_sum; r.k = (int)top_k; r.bias = bias; r.scale = scale;
    r.sigmoid = (flags & CR_FLAG_ROUTE_SIGMOID) != 0; r.renorm = (flags & CR_FLAG_ROUTE_RENORM) != 0;
    r.ids = ids; r.weights = weights;
    return from_hip(convrot::launch_route_experts(r, (int)dtype, stream));
}

size_t cr_experts_plan_workspace_bytes(int64_t T, int64_t top_k, int64_t E)
{
    return check_slots(T, top_k, 0, E) == CR_OK && T > 0 ? plan_bytes(T * top_k, E) : 0;
}

cr_status cr_experts_plan(const int32_t *ids, int64_t T, int64_t top_k, int64_t first, int64_t E, int32_t *offsets,
                          int32_t *rows, void *workspace, size_t ws_bytes, hipStream_t stream)
{
    cr_status s = check_slots(T, top_k, first, E);
    if (s != CR_OK) return s;
    if (!offsets || (T > 0 && (!ids || !rows))) return CR_ERR_INVALID_ARG;
    if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4)) return CR_ERR_MISALIGNED;
    const size_t need = T > 0 ? plan_bytes(T * top_k, E) : 0;
    if (need > 0) {
        if (!workspace) return CR_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
        if (ws_bytes < need) return CR_ERR_TOO_LARGE;
    }
    if ((s = current_device_ok()) != CR_OK) return s;
    return from_hip(convrot::launch_experts_plan(plan_launch(ids, T * top_k, first, E, offsets, rows, workspace), stream));
}

cr_status cr_gemm_s8s4_experts(const int8_t *a_s8, int64_t lda, const float *a_scale, int64_t M,
                               const uint8_t *b_s4, int64_t ldb, int64_t b_stride, const float *b_scale,
                               const float *bias, const int32_t *offsets, const int32_t *rows, int64_t S, int64_t E,
                               int64_t N, int64_t K_pad, int64_t gather, void *c, cr_dtype c_dtype, int64_t ldc,
                               uint32_t flags, hipStream_t stream)
{
    cr_status s = check_experts_gemm(a_s8, lda, a_scale, M, b_s4, ldb, b_stride, b_scale, bias, offsets, rows, S, E, N,
                                     K_pad, gather, c, c_dtype, ldc, flags);
    if (s != CR_OK || S == 0 || N == 0 || M == 0) return s;
    if ((s = current_device_ok()) != CR_OK) return s;
    return from_hip(convrot::launch_gemm_experts(
        experts_gemm(a_s8, lda, a_scale, M, b_s4, ldb, b_stride, b_scale, bias, offsets, rows, S, E, N, K_pad, gather,
                     (flags & CR_FLAG_EXPERTS_SCATTER) != 0, c, ldc),
        (int)c_dtype, (flags & CR_FLAG_EXPERTS_SWIGLU) != 0, stream));
}

cr_status cr_experts_combine(const void *y, cr_dtype dtype, int64_t ld_y, const float *weights, const int32_t *ids,
                             int64_t T, int64_t top_k, int64_t first, int64_t E, int64_t N, const void *residual,
                             int64_t ld_res, void *out, int64_t ld_out, hipStream_t stream)
{
    cr_status s = check_combine(y, dtype, ld_y, weights, ids, T, top_k, first, E, N, residual, ld_res, out, ld_out);
    if (s != CR_OK || T == 0 || N == 0) return s;
    if ((s = current_device_ok()) != CR_OK) return s;
    return from_hip(convrot::launch_experts_combine(
        combine_launch(y, ld_y, weights, ids, T, top_k, first, E, N, residual, ld_res, out, ld_out), (int)dtype, stream));
}

size_t cr_mlp_experts_w4a8_workspace_bytes(int64_t T, int64_t top_k, int64_t E, int64_t F, int64_t N, cr_dtype dtype)
{
    if (check_slots(T, top_k, 0, E) != CR_OK || T < 1 || F < 1 || N < 1 || N > kMostExpertCols || !is_float(dtype) ||
        F > CR_MAX_K_PAD || pad256(F) > CR_MAX_K_PAD)
        return 0;
    return plan_experts_layer(T, top_k, E, F, N, dtype).bytes;
}

cr_status cr_mlp_experts_w4a8(const int8_t *a_s8, int64_t lda, const float *a_scale, int64_t T, int64_t K_pad,
                              const int32_t *ids, const float *weights, int64_t top_k, int64_t first, int64_t E,
                              const uint8_t *w1, int64_t ld1, int64_t stride1, const float *scale1,
                              const float *bias1, int64_t F, const uint8_t *w2, int64_t ld2, int64_t stride2,
                              const float *scale2, const float *bias2, int64_t N, const void *residual,
                              int64_t ld_res, void *out, cr_dtype dtype, int64_t ld_out, void *workspace,
                              size_t ws_bytes, uint32_t flags, hipStream_t stream)
{
    if (!is_float(dtype)) return CR_ERR_UNSUPPORTED_DTYPE;
    cr_status s = check_slots(T, top_k, first, E);
    if (s != CR_OK) return s;
    if (check_flags(flags) != CR_OK || F < 1 || N < 0) return CR_ERR_INVALID_ARG;
    if (F > CR_MAX_K_PAD || pad256(F) > CR_MAX_K_PAD || N > kMostExpertCols) return CR_ERR_TOO_LARGE;
    const ExpertsPlan p = plan_experts_layer(T, top_k, E, F, N, dtype);
    const bool any = T > 0 && N > 0;
    // addresses of the workspace, or (an empty layer: nothing is enqueued) none
    int8_t *const ws = static_cast<int8_t *>(any ? workspace : nullptr);
    if (any) {
        if (!workspace) return CR_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return CR_ERR_MISALIGNED;
        if (ws_bytes < p.bytes) return CR_ERR_TOO_LARGE;
        if (!ids) return CR_ERR_INVALID_ARG;
    }
    auto at = [&](size_t off) { return any ? ws + off : nullptr; };
    int32_t *offsets = reinterpret_cast<int32_t *>(at(p.off_offsets));
    int32_t *rows = reinterpret_cast<int32_t *>(at(p.off_rows));
    void *h = at(p.off_h), *y = at(p.off_y);
    int8_t *q = at(p.off_q);
    float *q_scale = reinterpret_cast<float *>(at(p.off_scale));
    // validate every call before enqueueing anything; without columns the first product is checked too
    const int64_t S = any ? p.S : 0;
    s = check_experts_gemm(a_s8, lda, a_scale, T, w1, ld1, stride1, scale1, bias1, offsets, rows, S, E, 2 * F, K_pad,
                           top_k, h, dtype, p.ld_h, CR_FLAG_EXPERTS_SWIGLU);
    if (s != CR_OK) return s;
    s = check_act(h, dtype, p.ld_h, S, F, F, q, p.F_pad, q_scale, flags);
    if (s != CR_OK) return s;
    s = check_experts_gemm(q, p.F_pad, q_scale, S, w2, ld2, stride2, scale2, bias2, offsets, rows, S, E, N, p.F_pad, 0, y,
                           dtype, p.ld_y, CR_FLAG_EXPERTS_SCATTER);
    if (s != CR_OK) return s;
    s = check_combine(y, dtype, p.ld_y, weights, ids, any ? T : 0, top_k, first, E, N, residual, ld_res, out, ld_out);
    if (s != CR_OK || !any) return s;
    if ((s = current_device_ok()) != CR_OK) return s;
    const bool tp = (flags & CR_FLAG_FORCE_TWO_PASS) != 0, tr = (flags & CR_FLAG_BLOCK_TRANSPOSED) != 0;
    // Few slots: the products sort them themselves and leave the rows between them in the slots' order; the
    // plan would cost a launch (one token: 3.6 us of 40).  The rows are independent: the same bits.
    const bool own_plan = S <= convrot::kOwnPlan;
    convrot::ExpertsGemm up = experts_gemm(a_s8, lda, a_scale, T, w1, ld1, stride1, scale1, bias1, offsets, rows, S, E, 2 * F,
                                           K_pad, top_k, own_plan, h, p.ld_h);
    convrot::ExpertsGemm down = experts_gemm(q, p.F_pad, q_scale, S, w2, ld2, stride2, scale2, bias2, offsets, rows, S, E, N,
                                             p.F_pad, own_plan ? 1 : 0, true, y, p.ld_y);
    if (own_plan) {
        up.ids = down.ids = ids;
        up.first = down.first = (int)first;
    }
    if (!own_plan &&
        convrot::launch_experts_plan(plan_launch(ids, S, first, E, offsets, rows, at(p.off_counts)), stream) != hipSuccess)
        return CR_ERR_LAUNCH;
    if (convrot::launch_gemm_experts(up, (int)dtype, true, stream) != hipSuccess) return CR_ERR_LAUNCH;
    if (own_plan && !tr && convrot::experts_row_fits(T, S, N, p.F_pad)) {
        // one token: the second product prepares its rows itself
        down.A = static_cast<const int8_t *>(h);
        down.lda = p.ld_h;
        down.K = (int)F;
        if (convrot::launch_experts_row(down, (int)dtype, stream) != hipSuccess) return CR_ERR_LAUNCH;
    } else {
        if (convrot::launch_quant_act(h, (int)dtype, p.ld_h, S, F, nullptr, q, p.F_pad, q_scale, tp, tr, stream) != hipSuccess)
            return CR_ERR_LAUNCH;
        if (convrot::launch_gemm_experts(down, (int)dtype, false, stream) != hipSuccess) return CR_ERR_LAUNCH;
    }
    return from_hip(convrot::launch_experts_combine(
        combine_launch(y, p.ld_y, weights, ids, T, top_k, first, E, N, residual, ld_res, out, ld_out), (int)dtype, stream));
}

}  // extern "C"
