// Internal launchers of the gfx950 kernels (argument checking happens in api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace convrot {

// output tile of one GEMM workgroup (rows of A = activation rows, rows of B = weight rows)
constexpr int64_t kGemmTileCols = 256;   // M direction
constexpr int64_t kGemmTileRows = 256;   // N direction (weight rows)

// dtype codes follow cr_dtype: 0 bf16, 1 fp16, 2 fp32, 3 int32 (GEMM output only)
// pre: optional [K] (or [F]) channel pre-scale, nullptr for none; transposed: codes in the
// block-transposed column order (see row_prep.hpp)
hipError_t launch_quant_act(const void *x, int dtype, int64_t ld_x, int64_t M, int64_t K, const float *pre,
                            int8_t *x_s8, int64_t ld_s8, float *x_scale, bool two_pass, bool transposed,
                            hipStream_t st);

hipError_t launch_quant_act_swiglu(const void *h, int dtype, int64_t ld_h, int64_t M, int64_t F,
                                   const float *pre, int8_t *x_s8, int64_t ld_s8, float *x_scale,
                                   bool two_pass, bool transposed, hipStream_t st);

// residual addition (r nullptr: none; sum nullptr: not kept), RMS norm and S8 preparation
hipError_t launch_quant_act_rmsnorm(const void *x, int dtype, int64_t ld_x, const void *r, int64_t ld_r, void *sum,
                                    int64_t ld_sum, const float *w, float eps, int64_t M, int64_t K, int8_t *x_s8,
                                    int64_t ld_s8, float *x_scale, bool two_pass, bool transposed, int cus,
                                    hipStream_t st);

hipError_t launch_swiglu(const void *h, int dtype, int64_t ld_h, int64_t M, int64_t F, float *out,
                         int64_t ld_out, hipStream_t st);

// W4A8: dense weight rows -> ConvRot256 -> packed 4-bit codes [N, ld_s4 bytes] + scales
hipError_t launch_quant_weight_w4(const void *w, int dtype, int64_t ld_w, int64_t N, int64_t K, uint8_t *w_s4,
                                  int64_t ld_s4, float *w_scale, bool two_pass, bool transposed, hipStream_t st);

// The same 4-bit weight rows as E2M3 fields [N, ld_f6 bytes] (ld_f6 >= 3 K_pad / 4)
hipError_t launch_quant_weight_e2m3(const void *w, int dtype, int64_t ld_w, int64_t N, int64_t K, uint8_t *w_f6,
                                    int64_t ld_f6, float *w_scale, bool two_pass, bool transposed, hipStream_t st);

// nibble-form 4-bit rows [N, ld_s4] -> the same codes as E2M3 fields (quads of ld_f6 bytes)
hipError_t launch_repack_w4_e2m3(const uint8_t *w_s4, int64_t ld_s4, int64_t N, int64_t K_pad, uint8_t *w_f6,
                                 int64_t ld_f6, hipStream_t st);

// W4A4: activation rows (swiglu: H [M, 2K], SwiGLU first) -> ConvRot256 -> packed 4-bit
// codes [M, ld_s4 bytes] + scales, the format of launch_quant_weight_w4
hipError_t launch_quant_act_w4(const void *x, int dtype, int64_t ld_x, bool swiglu, int64_t M, int64_t K,
                               uint8_t *x_s4, int64_t ld_s4, float *x_scale, bool two_pass, bool transposed,
                               hipStream_t st);
hipError_t launch_quant_act_e2m3(const void *x, int dtype, int64_t ld_x, bool swiglu, int64_t M, int64_t K,
                                 uint8_t *x_f6, int64_t ld_f6, float *x_scale, bool two_pass, bool transposed,
                                 hipStream_t st);

hipError_t launch_prep_weight(const uint8_t *codes, int64_t ld_codes, const uint8_t *sf, int64_t ld_sf,
                              const float *g, int64_t n_rows, int64_t K, int8_t *w_s8, int64_t ld_s8,
                              float *w_scale, bool two_pass, bool transposed, hipStream_t st);

// bias: optional [N] FP32 bias added in the epilogue, nullptr for none (not with int32 out)
hipError_t launch_gemm_s8(const int8_t *A, int64_t lda, const float *sa, const int8_t *B, int64_t ldb,
                          const float *sb, const float *bias, int64_t M, int64_t N, int64_t K_pad, void *C,
                          int out_dtype, int64_t ldc, hipStream_t st);

// W4A8: S8 activation x packed 4-bit weight (the layout of launch_quant_weight_w4), same
// epilogue as launch_gemm_s8; ldb in bytes
hipError_t launch_gemm_s8s4(const int8_t *A, int64_t lda, const float *sa, const uint8_t *B, int64_t ldb,
                            const float *sb, const float *bias, int64_t M, int64_t N, int64_t K_pad, void *C,
                            int out_dtype, int64_t ldc, hipStream_t st);

// W4A4: packed 4-bit activation x packed 4-bit weight, same epilogue; lda, ldb in bytes
hipError_t launch_gemm_s4s4(const uint8_t *A, int64_t lda, const float *sa, const uint8_t *B, int64_t ldb,
                            const float *sb, const float *bias, int64_t M, int64_t N, int64_t K_pad, void *C,
                            int out_dtype, int64_t ldc, hipStream_t st);

// W4A4 on the 6-bit matrix cores: two E2M3-field operands (lda, ldb in bytes), same epilogue
hipError_t launch_gemm_e2m3(const uint8_t *A, int64_t lda, const float *sa, const uint8_t *B, int64_t ldb,
                            const float *sb, const float *bias, int64_t M, int64_t N, int64_t K_pad, void *C,
                            int out_dtype, int64_t ldc, hipStream_t st);

// row maximum a = max |rotated row| of NVFP4 weight rows (no codes)
hipError_t launch_weight_amax(const uint8_t *codes, int64_t ld_codes, const uint8_t *sf, int64_t ld_sf,
                              const float *g, int64_t n_rows, int64_t K, float *amax, bool two_pass,
                              hipStream_t st);

// decode-inside-GEMM over NVFP4 weights with given row maxima (transposed: order of A)
hipError_t launch_gemm_nvfp4_fused(const int8_t *A, int64_t lda, const float *sa, const uint8_t *codes,
                                   int64_t ld_codes, const uint8_t *sf, int64_t ld_sf, const float *g,
                                   const float *amax, const float *bias, int64_t M, int64_t N, int64_t K,
                                   void *C, int out_dtype, int64_t ldc, bool transposed, hipStream_t st);

// the 8-bit cache (kv8.hpp) and its page table
struct Kv8Ptrs {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    int64_t n_pages;
    const int32_t *table;
    int64_t ld_table;
};

// rotary embedding, per-head norm and append to the cache (dtype 0 bf16, 1 fp16; D 64 or 128)
struct RopeLaunch {
    const void *qkv;
    int dtype;
    int64_t ld_qkv;
    void *q_out;
    int64_t ld_q;
    const float *q_weight, *k_weight;
    float eps;
    const int32_t *pos;
    int64_t ld_pos;
    int n_axes;
    const double *freq;
    const int32_t *axis;
    int interleaved;
    int64_t T, B, max_new;
    const int32_t *cu, *kv_lens;
    int Hq, Hkv, D;
    Kv8Ptrs cache;
    int cus;
};
hipError_t launch_rope_append_kv8(const RopeLaunch &r, hipStream_t st);

// attention over the cache: which kernel runs and how the work is split (attn_kv8.hip).  A block is
// a run of query rows of one sequence and key/value head.
struct AttnPlan {
    bool few;                // few query rows a kv head: one wave holds a block's
    int64_t row_blocks;      // blocks a sequence and kv head
    int64_t whole, tail;     // blocks that one workgroup does, and blocks split over the cache
    int64_t splits, pages_per_split;
    int64_t part_rows;       // rows of partial results of one split,
    bool by_token;           // one for each token and head of the batch, or for each row of the split blocks
    int join_waves;          // waves that join a row
    int64_t join_groups;     // workgroups of the join
    size_t off_ml, bytes;    // workspace: partial outputs, then (maximum, sum) pairs
};
// workgroups of 256 threads that a dispatch's 32-bit work-item count allows
constexpr int64_t kMostBlocks = (int64_t)(UINT32_MAX / 256);
AttnPlan plan_attn_kv8(int64_t T, int64_t B, int64_t max_q, int64_t max_kv, int Hq, int Hkv, int D, int cus);

struct AttnLaunch {
    const void *q;
    int dtype;
    int64_t ld_q;
    void *out;
    int64_t ld_out;
    int64_t T, B;
    const int32_t *cu, *kv_lens;
    int Hq, Hkv, D;
    Kv8Ptrs cache;
    float sm_scale;
    int causal;
    void *workspace;
    AttnPlan plan;
};
hipError_t launch_attn_kv8(const AttnLaunch &l, hipStream_t st);

}  // namespace convrot
