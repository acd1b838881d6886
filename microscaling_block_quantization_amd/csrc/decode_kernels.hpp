// decode_kernels.hpp -- launch interface between the C ABI (api.hip) and the
// kernels of one decode step: products with 4-bit weights, the norm and
// rotation of query and key heads, the paged cache and its attention.
// Internal to libmx.so.
#pragma once
#include "mx_kernels.hpp"

namespace mxk {

// HIP takes fewer than 2^32 threads along a grid's axis.  A launcher returns
// this, with nothing launched, where a call would need more.
constexpr hipError_t TOO_LARGE = hipErrorInvalidConfiguration;
inline bool grid_ok(int64_t blocks, int threads) { return blocks * threads < (int64_t)1 << 32; }

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
// a division of numbers below 2^31 as a multiply and a shift
struct Div {
    uint32_t mul;
    int shift;
};
struct CacheWrite {
    KvCache c;
    const void *k, *v;
    int64_t k_ts, k_hs, v_ts, v_hs;
    const int64_t* slots;
    int64_t tokens;
    int rule;                      // E8M0 exponent rule
    float tau;
    Div per_token, page_div;       // set by the launcher: by the heads, by the page size
    int page_shift;                // its logarithm where it is a power of two, else -1
};
hipError_t launch_cache_write(CacheWrite p, bool in_bf16, hipStream_t s);

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
    Div page_div;                  // set by the launcher
};
// How a call is split: waves per workgroup; 0, or the workgroups that share the
// tokens of all sequences for each key-value head and 16 query heads
struct AttendPlan {
    int waves, workers;
};
AttendPlan attend_plan(const KvCache& c, int64_t batch, int q_heads, int64_t cols);
// Most slots per query head (workers + sequences, 0 without workers) of any call
// of at most this batch and these columns
int64_t attend_slots(const KvCache& c, int64_t batch, int q_heads, int64_t cols);
bool attend_dim_ok(int dim);
hipError_t launch_attend(AttendParams p, bool q_bf16, hipStream_t s);

}  // namespace mxk
