// logprobs.hip -- log probabilities of given tokens, entropy and the likeliest
// alternatives of rows of logits, and the gradient of the first two.
//
// Mathematics.  With m = max z, S = sum e^(z - m) and W = sum e^(z - m) (z - m):
//   lse = m + ln S,  log p_j = (z_j - m) - ln S,  H = -sum p ln p = ln S - W / S,
// and (m, S, W) of disjoint parts join by S' = e^(m - m') S, W' = e^(m - m')
// (W + (m - m') S).  One pass over the logits, memory bound.  The gradient is
//   dz_j = g (1[j = target] - p_j) - g_H p_j (ln p_j + H).
//
// Top alternatives.  A workgroup holds a segment of the row in registers, 16 KB.
// The k-th largest of its 256 lanes' maxima bounds the k-th largest element from
// below, and few elements besides the k largest reach it, so those are gathered
// in LDS and ranked by counting.  The bound is found by bisection over the
// values' order-preserving integers, each step four ballots.
//
// Bound and measured.  Large launches: memory; the gradient of 4096 x 131072 bf16
// 372 us, 5.8 TB/s read and written, of 333 x 50001 fp32 (rows at every
// alignment) 21 us.  64 rows of 131072 bf16 with 20 alternatives: 14.2 us and 4.6
// for the join, one round of workgroups whose load, exponentials, bisection and
// ranking follow each other.  Segments of 32 KB there 26 us, bisection over all
// integers instead of the lanes' range 15.2; the join by ranking every key 6.5,
// by bisection 8.8, by binary search in the splits' lists 14.5.  Without
// alternatives 4096 x 131072 bf16 takes 221 us, 4.9 TB/s, and 333 x 50001 fp32
// 15.9 and 3.9 for the join.
//
// Rounding.  An exponential's argument is one fp32 product with log2 e, a
// logarithm the hardware's times ln 2.  Against 64 bits (rms, of 64 x 131072 bf16
// and 333 x 50001 fp32) log p is off by 5 10^-8 of itself and the entropy by 6.6
// 10^-8; the elementary form in fp32 by 15 and 5.6.  Carrying the product's error
// along takes the entropy's from 5.7 to 4.4 in bf16, not at all in fp32, and the
// 14.2 us to 19.8; the last sums and logarithm in 64 bits leave it within a tenth.
#include "decode_kernels.hpp"

namespace mxk {
using namespace mxd;

namespace {

typedef float f2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

constexpr int LT = 256, NV = 4;                       // threads; 16-byte pieces of a lane in a segment
constexpr int EASY = 512;                             // candidates gathered without care for ties
constexpr float FAR = -1e20f;                         // a distance whose exponential is 0 and whose products stay finite
constexpr float LOG2E = 1.44269504088896340736f, LN2 = 0.69314718055994530942f;

template <bool BF>
struct Row {
    static constexpr int PER = BF ? 8 : 4, ES = BF ? 2 : 4;
    const char* at;            // the row's first element, rounded down to 16 bytes
    int shift;                 // elements between there and the row's first
    int64_t vocab, safe;       // pieces below `safe` can be read whole
    __device__ Row(const void* z, int64_t t, int64_t tokens, int64_t ld, int64_t v) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(z) + (uintptr_t)(t * ld * ES);
        at = reinterpret_cast<const char*>(a & ~(uintptr_t)15);
        shift = (int)(a & 15) / ES;
        vocab = v;
        // the tensor ends where its last row does
        safe = ((tokens - 1 - t) * ld + v + shift) / PER;
    }
    __device__ int64_t pieces() const { return (vocab + shift + PER - 1) / PER; }
    // piece q; what is not the row's is anything
    __device__ u32x4 load(int64_t q) const {
        if (q < safe) return *reinterpret_cast<const u32x4*>(at + 16 * q);
        u32x4 o = {0u, 0u, 0u, 0u};
        const int64_t left = vocab + shift - q * PER;
#pragma unroll
        for (int e = 0; e < PER; e++)
            if (e < left) {
                if (BF) o[e / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(at)[q * PER + e] << (16 * (e & 1));
                else o[e % 4] = reinterpret_cast<const uint32_t*>(at)[q * PER + e];
            }
        return o;
    }
    __device__ static float value(u32x4 w, int e) {
        if (BF) return (e & 1) ? bf16hi(w[e / 2]) : bf16lo(w[e / 2]);
        return bitsf(w[e % 4]);
    }
    __device__ float one(int64_t j) const {
        const char* p = at + (shift + j) * ES;
        return BF ? bf16f(*reinterpret_cast<const uint16_t*>(p)) : *reinterpret_cast<const float*>(p);
    }
};

struct Triple {
    float m, s, w;
};
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * LOG2E); }
__device__ __forceinline__ Triple join(Triple a, Triple b) {
    const float m = fmaxf(a.m, b.m), ms = m == -INFINITY ? 0.f : m;
    const float da = fmaxf(a.m - ms, FAR), db = fmaxf(b.m - ms, FAR), fa = exp_of(da), fb = exp_of(db);
    return Triple{m, fa * a.s + fb * b.s, fa * (a.w + da * a.s) + fb * (b.w + db * b.s)};
}
__device__ __forceinline__ Triple wave_join(Triple t) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) t = join(t, Triple{__shfl_xor(t.m, o, 64), __shfl_xor(t.s, o, 64), __shfl_xor(t.w, o, 64)});
    return t;
}

__device__ __forceinline__ float first_of(float x) { return bitsf((uint32_t)__builtin_amdgcn_readfirstlane((int)fbits(x))); }

// An integer in the order of the values: at least 1, -0 as +0, NaN as -Inf
__device__ __forceinline__ uint32_t order_of(float z) {
    const uint32_t u = fbits(z != z ? -INFINITY : z + 0.0f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}
constexpr uint32_t LEAST = 0x007fffffu;               // of -Inf
__device__ __forceinline__ float value_of(uint32_t o) { return bitsf((o >> 31) ? o & 0x7fffffffu : ~o); }
// larger values first, then lower places
__device__ __forceinline__ uint64_t key_of(uint32_t order, uint32_t place) { return (uint64_t)order << 32 | (uint32_t)~place; }

// the largest of a wave's numbers, in lane 63, by lane moves in the vector unit
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MOVED(ctrl, rows) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xf, false))
    MOVED(0x111, 0xf);                                // by 1, 2, 4, 8 lanes of a row of 16
    MOVED(0x112, 0xf);
    MOVED(0x114, 0xf);
    MOVED(0x118, 0xf);
    MOVED(0x142, 0xa);                                // a row's last to the next row, then half a wave's
    MOVED(0x143, 0xc);
#undef MOVED
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// Bisection: from `lo` up, the largest value that at least k of the numbers (N
// a lane, the same in every wave) reach, or one that no more than `enough` do.
// `lo` itself if fewer than k reach it.  All of them reach the smallest.
template <int N>
__device__ __forceinline__ int reach(const uint32_t (&of)[N], uint32_t b) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; i++) n += __popcll(__ballot(of[i] >= b));
    return n;
}
template <int N>
__device__ __forceinline__ uint32_t narrow(const uint32_t (&of)[N], uint32_t lo, int k, int enough) {
    uint32_t most = of[0], least = of[0];
#pragma unroll
    for (int i = 1; i < N; i++) {
        most = max(most, of[i]);
        least = min(least, of[i]);
    }
    uint32_t hi = wave_max(most) + 1;                 // which none reaches; no order is 2^32 - 1
    lo = max(lo, ~wave_max(~least));
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int n = reach(of, mid);
        if (n >= k) {
            lo = mid;
            if (n <= enough) break;
        } else {
            hi = mid;
        }
    }
    return lo;
}
// a few more than k: each step of the bisection costs as much as ranking some
__device__ __forceinline__ int few_more(int k) { return k + k / 2 + 4; }

// Writes the k largest of n distinct keys in order.
__device__ __forceinline__ void rank_keys(const uint64_t* keys, int n, uint64_t* best, int k, int tid) {
    for (int i = tid; i < n; i += LT) {
        const uint64_t mine = keys[i];
        int r = 0;
        int j = 0;
        for (; j + 4 <= n; j += 4) r += (keys[j] > mine) + (keys[j + 1] > mine) + (keys[j + 2] > mine) + (keys[j + 3] > mine);
        for (; j < n; j++) r += keys[j] > mine;
        if (r < k) best[r] = mine;
    }
}

__device__ __forceinline__ void finish(const LogprobParams& p, int64_t t, Triple s, float target, bool counts) {
    const float ln = __builtin_amdgcn_logf(s.s) * LN2;
    const bool none = s.m == -INFINITY && s.s == 0.f;          // nothing is possible (a NaN leaves s a NaN)
    p.lse[t] = none ? -INFINITY : s.m + ln;
    p.logprob[t] = !counts ? 0.f : none ? -INFINITY : (target - s.m) - ln;
    p.entropy[t] = none ? 0.f : ln - s.w / s.s;
}
__device__ __forceinline__ void put_top(const LogprobParams& p, int64_t t, int i, uint64_t key, Triple s) {
    const bool none = s.m == -INFINITY && s.s == 0.f;
    p.top_ids[t * p.top + i] = (int64_t)(uint32_t)~(uint32_t)key;
    p.top_logprobs[t * p.top + i] = none ? -INFINITY : (value_of((uint32_t)(key >> 32)) - s.m) - __builtin_amdgcn_logf(s.s) * LN2;
}

// Workgroup `split` of a row takes `segments` segments of it; with one split it
// writes the row's outputs, else its triple and keys to the workspace.
template <bool BF, bool TOP>
__global__ __launch_bounds__(LT) void k_logprobs(LogprobParams p) {
    typedef Row<BF> R;
    constexpr int PER = R::PER, E = NV * PER;
    constexpr int CAP = TOP ? MOST_TOP * (E + 2) : 1;
    __shared__ uint64_t keys[CAP], best[TOP ? MOST_TOP : 1];
    __shared__ uint32_t lane_max[TOP ? LT : 1];
    __shared__ int found, sums[LT / 64];
    __shared__ Triple parts[LT / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x / (uint32_t)p.splits;
    const int split = (int)(blockIdx.x - (uint32_t)t * (uint32_t)p.splits);
    const R row(p.z, t, p.tokens, p.ld, p.vocab);
    const int64_t pieces = row.pieces();
    const int64_t q0 = (int64_t)split * p.segments * (LT * NV);
    Triple s = {-INFINITY, 0.f, 0.f};
    int held = 0;                                              // keys in best
    const int k = p.top;

    for (int seg = 0; seg < p.segments; seg++) {
        const int64_t base = q0 + (int64_t)seg * (LT * NV);
        if (base >= pieces) break;
        u32x4 raw[NV];
#pragma unroll
        for (int v = 0; v < NV; v++) {
            const int64_t q = base + v * LT + tid;
            raw[v] = q < pieces ? row.load(q) : u32x4{0u, 0u, 0u, 0u};
        }
        // place of element e of piece v in the row; an edge piece holds others' too
        auto place = [&](int v, int e) { return (base + v * LT + tid) * PER + e - row.shift; };
        const bool edge = base == 0 || base + LT * NV >= row.vocab / PER;
        float m = -INFINITY;
        uint64_t live = ~0ull;                                 // elements of the row, bit PER v + e
        if (edge) {
            live = 0;
#pragma unroll
            for (int v = 0; v < NV; v++)
#pragma unroll
                for (int e = 0; e < PER; e++) {
                    const int64_t j = place(v, e);
                    if (j >= 0 && j < row.vocab) live |= 1ull << (PER * v + e);
                }
        }
        auto z_of = [&](int v, int e) {
            const float z = R::value(raw[v], e);
            return !edge || (live >> (PER * v + e) & 1) ? z : -INFINITY;
        };
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int e = 0; e < PER; e++) m = fmaxf(m, z_of(v, e));
        const float ms = m == -INFINITY ? 0.f : m;
        float sum = 0.f, w = 0.f;
#pragma unroll
        for (int v = 0; v < NV; v++)
#pragma unroll
            for (int e = 0; e < PER; e++) {
                const float d = z_of(v, e) - ms, x = exp_of(d);
                sum += x;
                w += x * fmaxf(d, FAR);
            }
        s = join(s, Triple{m, sum, w});

        if constexpr (TOP) {
            __syncthreads();
            // the lane's largest as an order; 0 where it has no element
            lane_max[tid] = live ? order_of(m) : 0u;
            if (tid == 0) found = 0;
            __syncthreads();
            const uint32_t beat = held == k ? (uint32_t)(best[k - 1] >> 32) : 0u;      // candidates lie above
            uint32_t of[LT / 64];
#pragma unroll
            for (int i = 0; i < LT / 64; i++) of[i] = lane_max[64 * i + lane];
            if (reach(of, beat + 1)) {
                uint32_t lo = narrow(of, beat + 1, k, few_more(k));
                auto gather = [&](uint32_t least, int most) {  // keys of elements of at least `least`
                    const bool all = least <= LEAST;           // NaN too
                    const float z0 = all ? -INFINITY : value_of(least);
#pragma unroll
                    for (int v = 0; v < NV; v++)
#pragma unroll
                        for (int e = 0; e < PER; e++) {
                            const float z = R::value(raw[v], e);
                            if ((z >= z0 || all) && (!edge || (live >> (PER * v + e) & 1))) {
                                const int at = atomicAdd(&found, 1);
                                if (at < most) keys[at] = key_of(order_of(z), (uint32_t)place(v, e));
                            }
                        }
                };
                gather(lo, EASY);
                __syncthreads();
                int n = found;
                if (n > EASY) {
                    // Ties, mostly: the k-th largest itself, what lies above it (of
                    // fewer than k lanes), and of the elements equal to it the first
                    // k places.
                    lo = narrow(of, lo, k, 0);
                    __syncthreads();
                    if (tid == 0) found = 0;
                    __syncthreads();
                    gather(lo + 1, CAP);
                    __syncthreads();
                    n = found;
                    int ties = 0;
#pragma unroll
                    for (int v = 0; v < NV; v++) {
                        uint32_t mask = 0;
#pragma unroll
                        for (int e = 0; e < PER; e++)
                            if ((!edge || (live >> (PER * v + e) & 1)) && order_of(R::value(raw[v], e)) == lo) mask |= 1u << e;
                        const int c = __popc(mask);
                        int upto = c;
#pragma unroll
                        for (int o = 1; o < 64; o <<= 1) {
                            const int x = __shfl_up(upto, o, 64);
                            if (lane >= o) upto += x;
                        }
                        if (lane == 63) sums[wave] = upto;
                        __syncthreads();
                        int at = ties + upto - c, all = ties;
#pragma unroll
                        for (int i = 0; i < LT / 64; i++) {
                            if (i < wave) at += sums[i];
                            all += sums[i];
                        }
#pragma unroll
                        for (int e = 0; e < PER; e++)
                            if (mask >> e & 1) {
                                if (at < k) keys[n + at] = key_of(lo, (uint32_t)place(v, e));
                                at++;
                            }
                        ties = all;
                        __syncthreads();
                    }
                    n += ties < k ? ties : k;
                }
                // with what earlier segments left
                if (tid < held) keys[n + tid] = best[tid];
                n += held;
                __syncthreads();
                rank_keys(keys, n, best, k, tid);
                held = n < k ? n : k;
                __syncthreads();
            }
        }
    }

    s = wave_join(s);
    if (lane == 0) parts[wave] = s;
    __syncthreads();
    s = parts[0];
#pragma unroll
    for (int i = 1; i < LT / 64; i++) s = join(s, parts[i]);
    if (p.splits == 1) {
        if (tid == 0) {
            const int64_t target = p.targets[t];
            const bool in = target >= 0 && target < p.vocab;
            finish(p, t, s, in ? row.one(target) : 0.f, in);
        }
        if (TOP && tid < k) put_top(p, t, tid, best[tid], s);
    } else {
        const int64_t at = t * p.splits + split;
        if (tid == 0) reinterpret_cast<Triple*>(p.parts)[at] = s;
        if (TOP && tid < k) p.keys[at * k + tid] = tid < held ? best[tid] : 0ull;
    }
}

// Joins the splits of a row.  A split's keys are in order (0 where it has fewer):
// the ceil(k / j)-th largest of the splits' j-th keys has k keys that are no
// smaller, and for j twice k / splits few more, so those are ranked alone.
template <bool BF, bool TOP>
__global__ __launch_bounds__(LT) void k_logprobs_join(LogprobParams p) {
    __shared__ uint64_t keys[TOP ? MOST_KEYS : 1], best[TOP ? MOST_TOP : 1];
    __shared__ uint64_t least;
    __shared__ int found;
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, k = p.top, splits = p.splits, n = splits * k;
    constexpr int PER = TOP ? MOST_KEYS / LT : 1;
    uint64_t mine[PER];
    if constexpr (TOP) {
#pragma unroll
        for (int i = 0; i < PER; i++) mine[i] = tid + LT * i < n ? p.keys[t * n + tid + LT * i] : 0ull;
        if (tid == 0) {
            least = 1ull;                                      // no place without a key
            found = 0;
        }
    }
    const Triple* parts = reinterpret_cast<const Triple*>(p.parts) + t * splits;
    Triple s = {-INFINITY, 0.f, 0.f};
    for (int i = lane; i < splits; i += 64) s = join(s, parts[i]);
    for (int o = 1; o < splits && o < 64; o <<= 1)
        s = join(s, Triple{__shfl_xor(s.m, o, 64), __shfl_xor(s.s, o, 64), __shfl_xor(s.w, o, 64)});
    s = Triple{first_of(s.m), first_of(s.s), first_of(s.w)};           // lanes from `splits` on joined nothing
    if (tid == 0) {
        const Row<BF> row(p.z, t, p.tokens, p.ld, p.vocab);
        const int64_t target = p.targets[t];
        const bool in = target >= 0 && target < p.vocab;
        finish(p, t, s, in ? row.one(target) : 0.f, in);
    }
    if constexpr (TOP) {
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (tid + LT * i < n) keys[tid + LT * i] = mine[i];
        __syncthreads();
        const int j = (2 * k + splits - 1) / splits < k ? (2 * k + splits - 1) / splits : k, m = (k + j - 1) / j;
        for (int i = tid; i < splits; i += LT) {
            const uint64_t it = keys[i * k + j - 1];
            int r = 0;
#pragma unroll 4
            for (int x = 0; x < splits; x++) r += keys[x * k + j - 1] > it;
            if (r == m - 1 && it) least = it;
        }
        __syncthreads();
        const uint64_t bound = least;
        // the few go to the front of the keys' place, which everyone has read
        __syncthreads();
#pragma unroll
        for (int i = 0; i < PER; i++)
            if (mine[i] >= bound) keys[atomicAdd(&found, 1)] = mine[i];
        __syncthreads();
        rank_keys(keys, found, best, k, tid);
        __syncthreads();
        if (tid < k) put_top(p, t, tid, best[tid], s);
    }
}

// The gradient: pieces of a row in the order of the logits' 16 bytes.
template <bool BF>
__global__ __launch_bounds__(LT) void k_logprobs_back(LogprobBackParams p) {
    typedef Row<BF> R;
    constexpr int PER = R::PER, V = 4;
    const int64_t t = blockIdx.x / (uint32_t)p.splits;
    const int64_t split = blockIdx.x - (uint32_t)t * (uint32_t)p.splits;
    const R row(p.z, t, p.tokens, p.ld, p.vocab);
    const int64_t pieces = row.pieces(), base = split * (LT * V);
    const int64_t target = p.targets[t];
    const bool in = target >= 0 && target < p.vocab;
    const float lse = p.lse[t], h = p.entropy ? p.entropy[t] : 0.f;
    const bool none = lse == -INFINITY;                        // nothing was possible: no gradient
    const float gl = p.d_logprob && in && !none ? p.d_logprob[t] : 0.f, gh = p.d_entropy && !none ? p.d_entropy[t] : 0.f;
    char* out = static_cast<char*>(p.dz) + t * p.ld_dz * R::ES;
    const bool same = (reinterpret_cast<uintptr_t>(out) & 15) == (uintptr_t)(row.shift * R::ES);
    u32x4 raw[V];
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int64_t q = base + v * LT + threadIdx.x;
        raw[v] = q < pieces ? row.load(q) : u32x4{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
        const int64_t q = base + v * LT + threadIdx.x;
        if (q >= pieces) break;
        const int64_t j0 = q * PER - row.shift;
        const int at = target >= j0 && target < j0 + PER ? (int)(target - j0) : -1;
        float dz[PER];
#pragma unroll
        for (int e = 0; e < PER; e++) {
            const float d = none ? -INFINITY : R::value(raw[v], e) - lse, x = exp_of(d);
            dz[e] = -x * (gl + gh * (fmaxf(d, FAR) + h));
            if (e == at) dz[e] += gl;
        }
        if (same && j0 >= 0 && j0 + PER <= row.vocab) {
            u32x4 o;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                if (BF) {
                    const f2v xy = {dz[(2 * e) % PER], dz[(2 * e + 1) % PER]};
                    o[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(xy, bf2v));
                } else {
                    o[e] = fbits(dz[e % PER]);
                }
            }
            *reinterpret_cast<u32x4*>(out + j0 * R::ES) = o;
        } else {
#pragma unroll
            for (int e = 0; e < PER; e++) {
                if (j0 + e < 0 || j0 + e >= row.vocab) continue;
                if (BF) reinterpret_cast<uint16_t*>(out)[j0 + e] = bf16_rne(dz[e]);
                else reinterpret_cast<float*>(out)[j0 + e] = dz[e];
            }
        }
    }
}

template <bool BF, bool TOP>
hipError_t run(const LogprobParams& p, hipStream_t s) {
    if (!grid_ok(p.tokens * p.splits, LT)) return TOO_LARGE;
    k_logprobs<BF, TOP><<<(unsigned)(p.tokens * p.splits), LT, 0, s>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.splits == 1) return e;
    k_logprobs_join<BF, TOP><<<(unsigned)p.tokens, LT, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace

// Segments a row is cut into (16 KB each, an unaligned start included), and how
// many a workgroup takes: one while the launch does not fill the chip.
LogprobPlan logprob_plan(int64_t tokens, int64_t vocab, int64_t ld, int top, bool bf16) {
    const int per = bf16 ? 8 : 4, unaligned = tokens > 1 && ld % per ? per - 1 : 0;
    const int64_t size = LT * NV * per, segments = (vocab + unaligned + size - 1) / size;
    LogprobPlan o;
    int64_t splits = tokens >= 1024 ? 1 : 2048 / tokens;
    if (splits > segments) splits = segments;
    const int64_t most = top ? MOST_KEYS / top : MOST_KEYS;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    o.segments = (int)((segments + splits - 1) / splits);
    o.splits = (int)((segments + o.segments - 1) / o.segments);
    return o;
}
int64_t logprob_bytes(int64_t tokens, int64_t vocab, int top) {
    // splits x tokens: below 1024 tokens at most 2048 and the tokens times the segments, the most for fp32
    if (tokens < 1 || vocab < 1) return 0;
    const int64_t segments = (vocab + 3 + LT * NV * 4 - 1) / (LT * NV * 4), few = tokens < 1023 ? tokens : 1023;
    int64_t rows = 2048 + few;
    if (rows > few * segments) rows = few * segments;
    return rows * ((int64_t)sizeof(Triple) + 8 * top) + 8 * 32;
}

hipError_t launch_logprobs(const LogprobParams& p, bool bf16, hipStream_t s) {
    if (p.top) return bf16 ? run<true, true>(p, s) : run<false, true>(p, s);
    return bf16 ? run<true, false>(p, s) : run<false, false>(p, s);
}

hipError_t launch_logprobs_back(LogprobBackParams p, bool bf16, hipStream_t s) {
    const int64_t size = LT * 4 * (bf16 ? 8 : 4), n = (p.vocab + (bf16 ? 7 : 3) + size - 1) / size;
    if (n >= (int64_t)1 << 31 || !grid_ok(p.tokens * n, LT)) return TOO_LARGE;
    p.splits = (int)n;
    if (bf16) k_logprobs_back<true><<<(unsigned)(p.tokens * n), LT, 0, s>>>(p);
    else k_logprobs_back<false><<<(unsigned)(p.tokens * n), LT, 0, s>>>(p);
    return hipGetLastError();
}

}  // namespace mxk
