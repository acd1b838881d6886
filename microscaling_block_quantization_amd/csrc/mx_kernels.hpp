// mx_kernels.hpp -- launch interface between the C ABI (api.hip) and the
// kernel translation units.  Internal to libmx.so.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.hpp"

namespace mxk {

// Everything a quantization launch needs.  Device pointers except where noted.
struct QParams {
    const void* x;
    int64_t rows, cols, ld;        // ld in elements
    int in_bf16;
    uint8_t* codes;
    uint8_t* scales;
    uint16_t* offsets;
    uint8_t* macro;
    const float* tensor_scale;     // NVFP4 g, produced by the pre-pass
    const int32_t* ref_exp;        // E3M0 e_ref, produced by the pre-pass
    void* dq;                      // nullable
    int dq_bf16;
    mxd::StatPart* parts;          // nullable: one partial per workgroup
    float* amax_parts;             // pre-pass mode: one max per workgroup
    int elem, asym, scale, rule, round;
    int br, bc, had, macro_cols;
    float tau;
    uint64_t seed, off;
};

constexpr int NT = 256;   // threads per workgroup for the streaming kernels

// row blocks (block_rows == 1): generic kernel; returns number of workgroups
int64_t rows_grid(const QParams& p);
hipError_t launch_rows(const QParams& p, bool amax_only, hipStream_t s);
// the E2M1 / E8M0 / RTNE row path on the hardware FP4 converter
bool rows_fast_ok(const QParams& p);
int64_t rows_fast_grid(const QParams& p);   // upper bound of the grid launch_rows_fast uses
hipError_t launch_rows_fast(const QParams& p, hipStream_t s, int64_t* grid);
// Several tensors of one such format and input dtype in one launch.  The
// caller fills x, codes, scales, parts (when p.parts is set: room for nb
// partials) and nchunks (16-byte chunks of input, nonzero) of job[0, count);
// the launcher sets b0 and nb, the workgroups each job takes.  *grid: the
// workgroups launched.
constexpr int MANY_MAX = 8;
struct FastJob {
    const void* x;
    uint8_t* codes;
    uint8_t* scales;
    mxd::StatPart* parts;
    int64_t nchunks, b0, nb;
};
struct FastMany {
    FastJob job[MANY_MAX];
    int count;
};
hipError_t launch_rows_fast_many(const QParams& p, FastMany& m, hipStream_t s, int64_t* grid);
// MXFP8 rows (E4M3 / E5M2 elements, E8M0 scales on 1 x 32 blocks, to nearest,
// dense) on the hardware FP8 converter
bool rows_fp8_ok(const QParams& p);
int64_t rows_fp8_grid(const QParams& p);    // upper bound of the grid launch_rows_fp8 uses
hipError_t launch_rows_fp8(const QParams& p, hipStream_t s, int64_t* grid);
// MXFP6 rows (E2M3 / E3M2, E8M0 scales on 1 x 32 blocks, to nearest, dense)
// on the hardware FP6 pack converter
bool rows_fp6_ok(const QParams& p);
int64_t rows_fp6_grid(const QParams& p);    // upper bound of the grid launch_rows_fp6 uses
hipError_t launch_rows_fp6(const QParams& p, hipStream_t s, int64_t* grid);
// the other E2M1 round-to-nearest row formats on the hardware FP4 converter
// (fp8 block scales, block Hadamard rotation, macro-block scales)
bool rows_hw_ok(const QParams& p);
int64_t rows_hw_grid(const QParams& p);     // upper bound of the grid launch_rows_hw uses
hipError_t launch_rows_hw(const QParams& p, hipStream_t s, int64_t* grid);
// column (b x 1) and 2D (b x b) blocks
int64_t tiles_grid(const QParams& p);
hipError_t launch_tiles(const QParams& p, hipStream_t s);
// tensor abs-max pre-pass (after the rotation, if any): amax_grid bounds the
// number of per-workgroup maxima; launch_amax reports the number written
int64_t amax_grid(const QParams& p);
hipError_t launch_amax(const QParams& p, hipStream_t s, int64_t* grid);
// finalize: tensor scale / reference exponent from the per-workgroup maxima
hipError_t launch_tensor_scale(const float* parts, int64_t n, int scale_kind, float qmax,
                               float* tensor_scale, int32_t* ref_exp, hipStream_t s);
// finalize: statistics from per-workgroup partials, fixed order
hipError_t launch_stats_final(const mxd::StatPart* parts, int64_t n, int64_t nelem, void* out,
                              hipStream_t s);
// the same for up to MANY_MAX partial sets in one launch, one workgroup each
struct FinalJob {
    const mxd::StatPart* parts;
    int64_t n, nelem;
    void* out;
};
struct FinalMany {
    FinalJob job[MANY_MAX];
};
hipError_t launch_stats_final_many(const FinalMany& m, int count, hipStream_t s);
// dequantize
hipError_t launch_dequant(const QParams& p, hipStream_t s);
// QSNR partials between two tensors
int64_t qsnr_grid(int64_t n);
hipError_t launch_qsnr(int bf16, const void* a, const void* b, int64_t n, mxd::StatPart* parts,
                       hipStream_t s);
// block-scaled GEMM; element codes E2M1, E2M3 or E3M2 for either operand
bool gemm_elem_ok(int elem);
hipError_t launch_gemm(int ea, const uint8_t* a, const uint8_t* sa, int eb, const uint8_t* b, const uint8_t* sb,
                       void* c, int64_t M, int64_t N, int64_t K, int64_t ldc, int c_bf16, hipStream_t s,
                       const uint8_t* ma = nullptr, const uint8_t* mb = nullptr);
// LDS-staged kernel for E8M0 1 x 32 operands of any element pair, K % 128 == 0
// (ma / mb: UE4M3 macro-block scales per 1 x 128, E2M1 operands only; nullable)
hipError_t launch_gemm_lds(int ea, const uint8_t* a, const uint8_t* sa, int eb, const uint8_t* b, const uint8_t* sb,
                           void* c, int64_t M, int64_t N, int64_t K, int64_t ldc, int c_bf16, hipStream_t s,
                           const uint8_t* ma = nullptr, const uint8_t* mb = nullptr);
// E2M1 operands under E8M0 / UE4M3 / NVFP4 / UE5M3 scales on 1 x bc blocks
// (bc a multiple of 8), decoded to bf16; ta / tb: per-tensor scales or null;
// ma / mb: UE4M3 macro-block scales per 1 x 128 (E8M0 block scales on both
// operands, K % 128 == 0), nullable
bool gemm_upcvt_scale_ok(int scale);
hipError_t launch_gemm_upcvt(int sca, int bca, const uint8_t* a, const uint8_t* sa, const float* ta, int scb, int bcb,
                             const uint8_t* b, const uint8_t* sb, const float* tb, void* c, int64_t M, int64_t N,
                             int64_t K, int64_t ldc, int c_bf16, hipStream_t s, const uint8_t* ma = nullptr,
                             const uint8_t* mb = nullptr);

// ---- the decode step (matvec.hip, qk_rope.hip, attend.hip) --------------------
struct MatvecParams {
    const uint8_t* codes;          // n x k/2
    const uint8_t* scales;         // n x k / block
    const uint16_t* offsets;       // nullable: bf16, n x k / block
    const uint8_t* macro;          // nullable: UE4M3, n x k/128
    const float* tensor_scale;     // nullable
    int64_t n, k;
    int elem, scale, lgb;          // lgb: log2 of the block width
    const void* x;                 // tokens x k, row stride ldx
    int64_t tokens, ldx;
    int x_bf16;
    const void* bias;              // nullable, the dtype of x
    void* y;
    int64_t ldy;
    int y_bf16;
};
hipError_t launch_matvec(const MatvecParams& p, hipStream_t s);

// queries or keys of a norm-and-rotation launch; strides in elements
struct RopeSet {
    const void* x;                 // the input heads
    const void* g;                 // backward: the outputs' gradient
    void* y;                       // the output heads, or the inputs' gradient
    int64_t x_ts, x_hs, g_ts, g_hs, y_ts, y_hs;
    uint32_t heads;                // 0: no such set
    const void* w;                 // nullable
    float* dw;                     // backward, where w is set
    float* parts;                  // backward: partial sums of dw, one row per workgroup
    uint32_t b0, nb;               // set by the launcher: this set's workgroups
};
struct RopeParams {
    RopeSet set[2];
    int64_t tokens, table_rows;
    int dim, rot, adjacent, w_bf16;
    const float *cos, *sin;
    const int32_t* positions;
    float eps;
};
constexpr int ROPE_PARTS = 1024;   // most workgroups (and partial rows) per set of a backward launch
hipError_t launch_rope(RopeParams p, bool bf16, bool back, hipStream_t s);

// cache element kinds
enum { KV_BF16 = 0, KV_FP8 = 1, KV_FP4 = 2 };
struct KvCache {
    uint8_t *k, *v, *ks, *vs;      // ks, vs: E8M0 scales, null for KV_BF16
    int64_t pages;
    int page, heads, dim, kind;
};
struct CacheWrite {
    KvCache c;
    const void *k, *v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    const int64_t* slots;
    int64_t tokens;
    int rule;                      // E8M0 exponent rule
    float tau;
};
hipError_t launch_cache_write(const CacheWrite& p, bool in_bf16, hipStream_t s);

struct AttendParams {
    KvCache c;
    const void* q;
    int64_t q_ts, q_hs;
    void* o;
    int64_t o_ts, o_hs;
    int64_t batch;
    int q_heads;
    const int32_t* table;
    int64_t cols, table_stride;
    const int32_t* lengths;
    float scale;
    float* lse;                    // nullable
    float* parts;                  // with workers: [q head][worker + sequence][dim] sums, then [..][2] max and sum
    int waves, workers;            // of the plan
    uint32_t page_mul;             // t / page = (t * page_mul) >> page_shift for t < 2^31
    int page_shift;
};
// How a call is split: waves per workgroup; 0, or the workgroups that share the
// tokens of all sequences for each key-value head and 16 query heads
struct AttendPlan {
    int waves, workers;
};
AttendPlan attend_plan(const KvCache& c, int64_t batch, int q_heads, int64_t cols);
bool attend_dim_ok(int dim);
hipError_t launch_attend(AttendParams p, bool q_bf16, hipStream_t s);

}  // namespace mxk
