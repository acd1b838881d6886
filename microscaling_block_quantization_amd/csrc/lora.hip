// lora.hip -- low-rank adapters of many requests beside a shared projection:
// y[t] = base[t] + s_a B_a (A_a x[t]), a the adapter that token t names.
//
// Mathematics.  Two products with a thin middle: h = A x (rank values a token)
// and B h.  Tokens come in tiles of 16, the columns of the 16 x 16 matrix
// instruction, whose rows are ranks (first product) or outputs (second).
// Columns are independent, so a tile whose tokens name several adapters runs
// once for each distinct one, the others' columns masked: a decode batch costs
// every adapter it uses once, a prompt of one adapter no more than a dense
// product, and tokens need no sorting.  bf16 operands: the 16 x 16 x 32 bf16
// instruction, h (fp32) as the exact sum of three bf16 parts side by side
// along K.  fp32 operands: the 16 x 16 x 4 fp32 instruction, products exact to
// its own rounding.
#include "decode_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

constexpr int TOK = 16;

// ids of the tile's tokens, one for each of 16 lanes (-1: none, or no such
// adapter), and the set of lanes that are the first with theirs
struct Ids {
    int id;
    uint32_t first;
};
__device__ __forceinline__ Ids tile_ids(const LoraParams& p, int64_t t0, int c) {
    Ids o;
    o.id = t0 + c < p.tokens ? p.ids[t0 + c] : -1;
    if (o.id < 0 || o.id >= p.count) o.id = -1;
    bool again = o.id < 0;
#pragma unroll
    for (int i = 0; i < TOK - 1; i++) again |= i < c && __builtin_amdgcn_readlane(o.id, i) == o.id;
    o.first = (uint32_t)__ballot(!again) & 0xffffu;
    return o;
}

// x as three bf16 parts, truncated (exact; Inf and NaN keep their first)
__device__ __forceinline__ uint16_t part3(float x, int part) {
    const uint32_t u = fbits(x);
    if ((u & 0x7f800000u) == 0x7f800000u) return part ? 0 : bf16_rne(x);
    const float r = x - bitsf(u & 0xffff0000u);
    const uint32_t v = fbits(r);
    return (uint16_t)((part == 0 ? u : part == 1 ? v : fbits(r - bitsf(v & 0xffff0000u))) >> 16);
}

__device__ __forceinline__ f4v mfma_bf16(u32x4 a, u32x4 b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
}
// the product of 16 K positions, four of a lane's each
__device__ __forceinline__ f4v mfma_f32(u32x4 a, u32x4 b, f4v c) {
#pragma unroll
    for (int e = 0; e < 4; e++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(bitsf(a[e]), bitsf(b[e]), c, 0, 0, 0);
    return c;
}

// ---------------------------------------------------------------------------
// h = A x.  Eight waves share K in steps of 64 bytes a lane, RT tiles of 16
// ranks each; a workgroup takes one of `splits` runs of K.  The waves' sums are
// added in LDS in their order, the runs' by the second product.
// ---------------------------------------------------------------------------
constexpr int SW = 8;

template <bool F32, int RT>
__global__ __launch_bounds__(64 * SW) void k_lora_down(LoraParams p) {
    constexpr int ES = F32 ? 4 : 2, PER = 64 / ES, STEP = 4 * PER;       // values a lane and a wave take at a time
    __shared__ __attribute__((aligned(16))) float red[SW][RT][256];
    const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    uint32_t rest = blockIdx.x;
    const int split = (int)(rest % (uint32_t)p.splits);
    rest /= (uint32_t)p.splits;
    const int turn = (int)(rest % (uint32_t)p.spread);                   // which of the tile's adapters, where they are spread
    rest /= (uint32_t)p.spread;
    const int r0 = (int)(rest % (uint32_t)p.rank_groups) * 16 * RT;
    const int64_t t0 = (int64_t)(rest / (uint32_t)p.rank_groups) * TOK;
    const Ids ids = tile_ids(p, t0, c);
    const int k = (int)p.k, steps = (k + STEP - 1) / STEP;
    const int from = (int)((int64_t)split * steps / p.splits), to = (int)((int64_t)(split + 1) * steps / p.splits);
    const int64_t tok = t0 + c < p.tokens ? t0 + c : p.tokens - 1;
    const char* x = static_cast<const char*>(p.x) + (tok * p.ldx + PER * g) * ES;

    f4v acc[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
    int seen = 0;
    for (uint32_t left = ids.first; left; left &= left - 1, seen++) {
        if (p.spread > 1 && seen != turn) continue;
        const int a = __builtin_amdgcn_readlane(ids.id, __builtin_ctz(left));
        const char* w[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) {
            const int r = r0 + 16 * i + c < p.rank ? r0 + 16 * i + c : p.rank - 1;
            w[i] = static_cast<const char*>(p.a) + (((int64_t)a * p.rank + r) * k + PER * g) * ES;
        }
        f4v sum[RT];
#pragma unroll
        for (int i = 0; i < RT; i++) sum[i] = f4v{0.f, 0.f, 0.f, 0.f};
        for (int s = from + wave; s < to; s += SW) {
            const int k0 = s * STEP, have = (k - k0 - PER * g) * ES / 16;      // 16-byte pieces of this lane's that exist
            u32x4 xv[4], wv[RT][4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const bool in = j < have;
                xv[j] = in ? *reinterpret_cast<const u32x4*>(x + (int64_t)k0 * ES + 16 * j) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < RT; i++)
                    wv[i][j] = in ? *reinterpret_cast<const u32x4*>(w[i] + (int64_t)k0 * ES + 16 * j) : u32x4{0u, 0u, 0u, 0u};
            }
#pragma unroll
            for (int j = 0; j < 4; j++)
#pragma unroll
                for (int i = 0; i < RT; i++) sum[i] = F32 ? mfma_f32(wv[i][j], xv[j], sum[i]) : mfma_bf16(wv[i][j], xv[j], sum[i]);
        }
#pragma unroll
        for (int i = 0; i < RT; i++)
            if (ids.id == a) acc[i] = sum[i];
    }
    if (p.spread > 1 && turn >= __builtin_popcount(ids.first)) return;       // the same in every wave
#pragma unroll
    for (int i = 0; i < RT; i++) *reinterpret_cast<f4v*>(&red[wave][i][c * 16 + 4 * g]) = acc[i];     // [token][rank]
    __syncthreads();
    int mine = 0;                                                        // the spread adapter's id
    if (p.spread > 1) {
        uint32_t left = ids.first;
        for (int i = 0; i < turn; i++) left &= left - 1;
        mine = __builtin_amdgcn_readlane(ids.id, __builtin_ctz(left));
    }
    for (int n = tid; n < 256 * RT; n += 64 * SW) {
        const int i = n % (16 * RT), t = n / (16 * RT);                  // rank, token
        const int id = __shfl(ids.id, t, 64);
        if (t0 + t >= p.tokens || r0 + i >= p.rank || id < 0 || (p.spread > 1 && id != mine)) continue;
        float v = 0.f;
#pragma unroll
        for (int q = 0; q < SW; q++) v += red[q][i / 16][t * 16 + i % 16];
        p.h[((int64_t)split * p.tokens + t0 + t) * p.rank + r0 + i] = v;
    }
}

// ---------------------------------------------------------------------------
// y = base + B h.  A wave takes NT tiles of 16 outputs, whose rows are dealt so
// that a lane ends with 4 NT consecutive outputs of its token, and goes down
// `run` tiles of tokens with B in registers while they name the same adapter.
// ---------------------------------------------------------------------------
constexpr int UW = 4;

template <bool BF, int N>
__device__ __forceinline__ void load_run(float (&o)[N], const void* p, int64_t at, int have, bool vec) {
    if (BF) {
        const uint16_t* x = static_cast<const uint16_t*>(p) + at;
        if (vec && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const uint2 w = *reinterpret_cast<const uint2*>(x + i);
                o[i] = bf16lo(w.x); o[i + 1] = bf16hi(w.x); o[i + 2] = bf16lo(w.y); o[i + 3] = bf16hi(w.y);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) o[i] = i < have ? bf16f(x[i]) : 0.f;
        }
    } else {
        const float* x = static_cast<const float*>(p) + at;
        if (vec && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const f4v w = *reinterpret_cast<const f4v*>(x + i);
                o[i] = w[0]; o[i + 1] = w[1]; o[i + 2] = w[2]; o[i + 3] = w[3];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) o[i] = i < have ? x[i] : 0.f;
        }
    }
}
template <int N>
__device__ __forceinline__ void store_run(const float (&o)[N], void* p, int64_t at, int have, bool vec, bool bf) {
    if (bf) {
        uint16_t* x = static_cast<uint16_t*>(p) + at;
        if (vec && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const f2v a = {o[i], o[i + 1]}, b = {o[i + 2], o[i + 3]};
                *reinterpret_cast<uint2*>(x + i) = make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf2v)),
                                                              __builtin_bit_cast(uint32_t, __builtin_convertvector(b, bf2v)));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (i < have) x[i] = bf16_rne(o[i]);
        }
    } else {
        float* x = static_cast<float*>(p) + at;
        if (vec && have >= N) {
#pragma unroll
            for (int i = 0; i < N; i += 4) *reinterpret_cast<f4v*>(x + i) = f4v{o[i], o[i + 1], o[i + 2], o[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < N; i++)
                if (i < have) x[i] = o[i];
        }
    }
}

// R8: runs of 8 ranks of a group (1, 2, 4 or 8), further groups of 64 in turn
template <bool F32, int R8, int NT>
__global__ __launch_bounds__(64 * UW) void k_lora_up(LoraParams p) {
    constexpr int ES = F32 ? 4 : 2, N = 4 * NT;
    // bf16: K slot 8 (4 j + g) holds run (4 j + g) % R8 of part (4 j + g) / R8;
    // fp32: slot 4 (4 j + g) the four ranks there
    constexpr int J = F32 ? (R8 + 1) / 2 : (3 * R8 + 3) / 4;
    constexpr int FR = F32 ? J : R8 <= 4 ? 1 : R8 / 4;                   // distinct pieces of B's row a lane holds
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * UW + wave) * 16 * NT;
    if (n0 >= p.n) return;
    const int64_t tiles = (p.tokens + TOK - 1) / TOK;
    const int64_t first = (int64_t)blockIdx.y * p.run, last = first + p.run < tiles ? first + p.run : tiles;
    const int64_t n = n0 + N * g;                                        // this lane's outputs
    const int have = (int)(p.n - n < N ? p.n - n : N);                   // may be negative
    const int groups = (p.rank + 8 * R8 - 1) / (8 * R8);

    u32x4 w[NT][FR];
    int held = -1;
    // B's rows of group q: row i of tile s is output n0 + N (i / 4) + 4 s + i % 4
    auto load_b = [&](int a, int q) {
#pragma unroll
        for (int s = 0; s < NT; s++) {
            const int64_t row = n0 + N * (c / 4) + 4 * s + c % 4;
            const char* b = static_cast<const char*>(p.b) + ((int64_t)a * p.n + (row < p.n ? row : p.n - 1)) * p.rank * ES;
#pragma unroll
            for (int f = 0; f < FR; f++) {
                const int r = q * 8 * R8 + (F32 ? 16 * f + 4 * g : R8 <= 4 ? 8 * (g % R8) : 32 * f + 8 * g);
                w[s][f] = r < p.rank ? *reinterpret_cast<const u32x4*>(b + r * ES) : u32x4{0u, 0u, 0u, 0u};
            }
        }
    };
    for (int64_t tile = first; tile < last; tile++) {
        const int64_t t0 = tile * TOK, tok = t0 + c < p.tokens ? t0 + c : p.tokens - 1;
        const Ids ids = tile_ids(p, t0, c);
        float base[N];
        if (p.base) {
            if (p.base_bf16) load_run<true>(base, p.base, tok * p.ld_base + n, have, p.vec_base);
            else load_run<false>(base, p.base, tok * p.ld_base + n, have, p.vec_base);
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) base[i] = 0.f;
        }
        f4v acc[NT];
#pragma unroll
        for (int s = 0; s < NT; s++) acc[s] = f4v{0.f, 0.f, 0.f, 0.f};
        const float scale = p.scales && ids.id >= 0 ? p.scales[ids.id] : 1.f;
        for (int q = 0; q < groups; q++) {
            // the token's h as columns
            u32x4 h[J];
#pragma unroll
            for (int j = 0; j < J; j++) {
                const int slot = 4 * j + g, part = F32 ? 0 : slot / R8;
                const int r = q * 8 * R8 + (F32 ? 4 * slot : 8 * (slot % R8));
                constexpr int V = F32 ? 4 : 8;
                float v[V];
#pragma unroll
                for (int e = 0; e < V; e++) v[e] = 0.f;
                if (ids.id >= 0 && part < 3 && r < p.rank)
                    for (int s = 0; s < p.splits; s++) {
                        const f4v* from = reinterpret_cast<const f4v*>(p.h + ((int64_t)s * p.tokens + tok) * p.rank + r);
#pragma unroll
                        for (int e = 0; e < V; e++) v[e] += from[e / 4][e % 4];
                    }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    if (F32) h[j][e] = fbits(v[e] * scale);
                    else h[j][e] = part3(v[(2 * e) % V] * scale, part) | (uint32_t)part3(v[(2 * e + 1) % V] * scale, part) << 16;
                }
            }
            for (uint32_t left = ids.first; left; left &= left - 1) {
                const int a = __builtin_amdgcn_readlane(ids.id, __builtin_ctz(left));
                if (a != held || groups > 1) {
                    load_b(a, q);
                    held = a;
                }
#pragma unroll
                for (int j = 0; j < J; j++) {
                    const u32x4 x = ids.id == a ? h[j] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int s = 0; s < NT; s++) {
                        if (F32) acc[s] = mfma_f32(w[s][j % FR], x, acc[s]);
                        else acc[s] = mfma_bf16(w[s][j % FR], x, acc[s]);
                    }
                }
            }
        }
        if (t0 + c < p.tokens && have > 0) {
#pragma unroll
            for (int i = 0; i < N; i++) base[i] += acc[i / 4][i % 4];
            store_run(base, p.y, tok * p.ldy + n, have, p.vec_y, p.y_bf16);
        }
    }
}

template <bool F32, int RT>
hipError_t down(const LoraParams& p, hipStream_t s) {
    const int64_t n = (p.tokens + TOK - 1) / TOK * p.rank_groups * p.spread * p.splits;
    if (!grid_ok(n, 64 * SW)) return TOO_LARGE;
    k_lora_down<F32, RT><<<(unsigned)n, 64 * SW, 0, s>>>(p);
    return hipGetLastError();
}
template <bool F32, int R8, int NT>
hipError_t up(const LoraParams& p, hipStream_t s) {
    const int64_t n = (p.n + 16 * NT * UW - 1) / (16 * NT * UW), tiles = (p.tokens + TOK - 1) / TOK;
    const dim3 grid((unsigned)n, (unsigned)((tiles + p.run - 1) / p.run));
    k_lora_up<F32, R8, NT><<<grid, 64 * UW, 0, s>>>(p);
    return hipGetLastError();
}
template <bool F32, int NT>
hipError_t up_rank(const LoraParams& p, hipStream_t s) {
    if (p.rank <= 8) return up<F32, 1, NT>(p, s);
    if (p.rank <= 16) return up<F32, 2, NT>(p, s);
    return p.rank <= 32 ? up<F32, 4, NT>(p, s) : up<F32, 8, NT>(p, s);
}
template <bool F32>
hipError_t both(LoraParams p, hipStream_t s) {
    p.rank_groups = (p.rank + 63) / 64;
    const hipError_t e = p.rank <= 16 ? down<F32, 1>(p, s) : p.rank <= 32 ? down<F32, 2>(p, s) : down<F32, 4>(p, s);
    if (e != hipSuccess) return e;
    return p.tokens <= TOK ? up_rank<F32, 1>(p, s) : up_rank<F32, 4>(p, s);
}

}  // namespace

// Runs of K for few tokens, whose first product is a chain of loads
constexpr int FEW = 64, MOST_SPLITS = 8;
int lora_splits(int64_t tokens, int64_t k) {
    if (tokens > FEW) return 1;
    const int64_t n = k / 1024;
    return (int)(n < 1 ? 1 : n > MOST_SPLITS ? MOST_SPLITS : n);
}
int64_t lora_rows(int64_t tokens) {
    const int64_t few = (tokens < FEW ? tokens : FEW) * MOST_SPLITS;
    return tokens > few ? tokens : few;
}

hipError_t launch_lora(LoraParams p, hipStream_t s) {
    const int64_t tiles = (p.tokens + TOK - 1) / TOK;
    p.splits = lora_splits(p.tokens, p.k);
    p.spread = p.tokens <= 1024 ? (int)(p.tokens < TOK ? p.tokens : TOK) : 1;
    if (p.spread > p.count) p.spread = p.count > 0 ? p.count : 1;
    // tiles of tokens a workgroup goes down: about 2048 workgroups
    const int64_t n = (p.n + 64 * UW - 1) / (64 * UW), run = tiles * n / 2048;
    p.run = (int)(run < 1 ? 1 : run > 64 ? 64 : run);
    if ((tiles + p.run - 1) / p.run > 65535) p.run = (int)((tiles + 65534) / 65535);
    return p.bf16 ? both<false>(p, s) : both<true>(p, s);
}

}  // namespace mxk
