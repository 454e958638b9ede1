// Routing to experts: which experts a token goes to and with which weights, the
// rows' order by expert, the gradient of the weights, and the rows' way to their
// experts and back.
//
// Choice.  Experts are ranked by a 64-bit key, the largest first: the value as a double,
// its lowest 11 bits given to the expert's number so that no two keys are equal and the
// lower number wins a tie.  Without a bias the value is the logit itself, which ranks as
// its score does; where keys are sums (a bias, or a group's two best) the scores are
// taken in fp64, so that which expert is chosen does not hang on how an fp32 score was
// rounded (the 42 bits that are left decide).  A token's LPT lanes hold VPL neighbouring
// experts each, so one wave routes 64 / LPT tokens.  A lane sorts its keys once, by
// fp64 minima and maxima; each of the top_k steps is then a maximum of the lanes' first
// keys (log2 LPT exchanges, four of them without LDS) and one lane's step to its next.
// 16384 tokens of 256 experts, 8 of them from 4 of 8 groups by sigmoid and bias: 27 us
// (softmax without a bias 15), and 9 for the rows' order, where reading the logits takes
// 3.6.  Latency at two waves a SIMD bounds it: the sixteen keys and scores of a lane take
// 241 registers, the waves issue in 29 % of their cycles and wait in 51 %.  12 us go to
// loads, sorting and first keys, 8 to scores in fp64, 4 to groups, 0.4 to each expert
// chosen; half as many experts a lane took 39 us.  The order's two launches wait in
// four fifths of their cycles.
//
// Order of rows.  Rows are sorted by expert and, within an expert, by token: a
// counting sort without atomics on memory.  In a block of up to 64 tokens every
// expert has one 64-bit word in LDS, token i's choices set bit i of their experts'
// words (an `or`, so their order does not matter), and a choice's place within the
// block is the number of bits below its own.  The blocks' counts are then summed over
// the blocks, expert by expert, and over the experts: by each block for itself, or in a
// launch of its own where that is many counts.
//
// Memory bounds the moves: a wave or more of lanes per token, 16 bytes a lane, a
// token read once for all its copies.  8192 tokens of 4096 values to 2 of 8 experts take
// 36 us, back with a residual 47 (5.7 TB/s in all); the gradient of the way back, 4096
// tokens of 2048 from 8 of 64, 70 us, 4.1 TB/s: it reads and writes rows in no order, and
// holds eight of them a lane (four and then four took 76).
#include <hip/hip_runtime.h>

#include "checks.h"
#include "vec.h"

namespace zs {
namespace {

constexpr int kRouteTokens = 64;   // tokens of a block: bits of an expert's word
constexpr int kGroupTokens = 16;   // the same where groups need LDS for every key
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 16;
constexpr int kMaxGroups = 64;

__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

struct RouteArgs {
    int64_t tokens, ldl;
    const void *logits;
    const float *bias;
    const uint8_t *active;
    int32_t *experts, *rows_of;
    float *weights;
    int64_t *offsets;
    int32_t *counts;  // blocks x experts
    int32_t *totals;  // experts
    float scale;
    int32_t n_experts, top_k, n_groups, top_groups, per_block;
    bool sigmoid, renorm, two, bf16, alone;  // two: a group's two best; alone: one block
};

// The key of expert e: values that are no number, and infinities, become numbers past
// all that fp32 holds, in order (NaN lowest); what is left out has the key -inf.
__device__ __forceinline__ double key_of(double x, int e)
{
    x += 0.0;  // -0 ranks as 0
    x = x == __builtin_inf() ? 1e300 : x == -__builtin_inf() ? -1e300 : x != x ? -1e301 : x;
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    return __longlong_as_double((long long)((u & ~2047ull) | (uint32_t)(u >> 63 ? e : 1024 - e)));
}

__device__ __forceinline__ int expert_of(double key)
{
    const uint64_t u = (uint64_t)__double_as_longlong(key);
    const int low = (int)(u & 2047);
    return u >> 63 ? low : 1024 - low;
}

// Descending order of N values, by Batcher's odd-even merges: static places only.
template <int N>
__device__ __forceinline__ void sort_down(double (&x)[N])
{
#pragma unroll
    for (int p = 1; p < N; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i)
                    if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
                        const double a = x[i + j], b = x[i + j + q];
                        x[i + j] = __builtin_fmax(a, b);
                        x[i + j + q] = __builtin_fmin(a, b);
                    }
}

// x of another lane, so that after the steps 1, 2, 4, ... N / 2 of a reduction its N
// neighbouring lanes agree: within 16 lanes by permutation (neighbours, pairs, and
// the mirrors of 8 and 16), which costs a move, then through LDS.
template <int STEP, class T>
__device__ __forceinline__ T other(T x)
{
    if constexpr (STEP >= 16) {
        return __shfl_xor(x, STEP, 64);
    } else {
        constexpr int CTRL = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
        int w[sizeof(T) / 4];
        __builtin_memcpy(w, &x, sizeof(T));
#pragma unroll
        for (unsigned i = 0; i < sizeof(T) / 4; ++i)
            w[i] = __builtin_amdgcn_mov_dpp(w[i], CTRL, 0xf, 0xf, true);
        __builtin_memcpy(&x, w, sizeof(T));
        return x;
    }
}

template <int N, int STEP = 1>
__device__ __forceinline__ double max_over(double x)
{
    if constexpr (STEP < N)
        return max_over<N, 2 * STEP>(__builtin_fmax(x, other<STEP>(x)));
    return x;
}

template <int N, int STEP = 1>
__device__ __forceinline__ float max_over(float x)
{
    if constexpr (STEP < N)
        return max_over<N, 2 * STEP>(fmaxf(x, other<STEP>(x)));
    return x;
}

template <int N, int STEP = 1, class T>
__device__ __forceinline__ T sum_over(T x)
{
    if constexpr (STEP < N)
        return sum_over<N, 2 * STEP>(x + other<STEP>(x));
    return x;
}

// VPL neighbouring logits from expert e0 on; -inf past the last.
template <int VPL>
__device__ __forceinline__ void load_logits(const void *logits, bool bf16, int64_t at, int e0, int E,
                                            float (&z)[VPL])
{
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        z[v] = -__builtin_inff();
    if constexpr (VPL >= 8) {
        if (e0 + VPL <= E) {
#pragma unroll
            for (int v = 0; v < VPL; v += 8) {
                float w[8];
                load8(logits, bf16, at + e0 + v, true, 8, w);
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    z[v + k] = w[k];
            }
            return;
        }
    }
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        if (e0 + v < E)
            z[v] = bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(logits)[at + e0 + v] << 16)
                        : static_cast<const float *>(logits)[at + e0 + v];
}

// e^x for x <= 0 (and NaN) in fp64, within 2^-50: 2^n e^r with |r| <= ln 2 / 2, e^r by its
// Taylor sum of degree 13 (the next term is below 2^-57).  r = x - n ln 2 takes ln 2 in two
// parts (Cody and Waite's reduction): its first 33 bits, of which n times is exact, and
// what is left, rounded.  Below -700 it is e^-700.
__device__ __forceinline__ double exp_below(double x)
{
    x = x < -700.0 ? -700.0 : x;
    const double n = __builtin_rint(x * 1.4426950408889634);
    const double r = __builtin_fma(-n, 1.9082149292705877e-10, __builtin_fma(-n, 0.6931471803691238, x));
    // the factorials' inverses in scalar registers, or each takes a move of its own
    double c[12] = {1.0 / 6227020800.0, 1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0,
                    1.0 / 40320.0,      1.0 / 5040.0,      1.0 / 720.0,      1.0 / 120.0,     1.0 / 24.0,
                    1.0 / 6.0,          0.5};
    double p = c[0];
#pragma unroll
    for (int i = 1; i < 12; ++i) {
        asm("" : "+s"(c[i]));
        p = __builtin_fma(p, r, c[i]);
    }
    p = __builtin_fma(p, r, 1.0);
    p = __builtin_fma(p, r, 1.0);
    return __builtin_ldexp(p, (int)n);
}
__device__ __forceinline__ float exp_below(float x) { return __expf(x); }

// 1 / x for x in [1, 2^11]: the hardware's reciprocal and two steps of Newton's.
__device__ __forceinline__ double inverse(double x)
{
    double y = __builtin_amdgcn_rcp(x);
    y = __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
    return __builtin_fma(__builtin_fma(-x, y, 1.0), y, y);
}
__device__ __forceinline__ float inverse(float x) { return 1.0f / x; }

template <class T>
__device__ __forceinline__ T sigmoid_of(float z)
{
    const T e = exp_below((T)-__builtin_fabsf(z)), y = inverse((T)1 + e);
    return z < 0.0f ? e * y : y;
}

// A token's softmax: the largest logit and 1 / sum (0 for a row of -inf alone, whose
// scores are 0).
template <class T>
struct Softmax {
    float most;
    T inv;
    __device__ __forceinline__ T numerator(float z) const
    {
        const T e = exp_below((T)z - (T)most);
        return z == -__builtin_inff() ? (T)0 : e;
    }
};

// The scores of a token's logits (0 past the last).
template <int LPT, int VPL, class T>
__device__ __forceinline__ Softmax<T> scores(const float (&z)[VPL], bool sigmoid, int e0, int E, T (&p)[VPL])
{
    Softmax<T> m = {0.0f, (T)0};
    if (sigmoid) {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            p[v] = sigmoid_of<T>(z[v]);
            if constexpr (sizeof(T) == 8)  // two at a time: more side by side take more registers than there are
                if (v & 1)
                    __builtin_amdgcn_sched_barrier(0);
            if (e0 + v >= E)
                p[v] = 0;
        }
        return m;
    }
    m.most = z[0];
#pragma unroll
    for (int v = 1; v < VPL; ++v)
        m.most = fmaxf(m.most, z[v]);
    m.most = max_over<LPT>(m.most);
    T sum = 0;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        p[v] = m.numerator(z[v]);
        if constexpr (sizeof(T) == 8)
            if (v & 1)
                __builtin_amdgcn_sched_barrier(0);
        sum += p[v];
    }
    sum = sum_over<LPT>(sum);
    m.inv = sum == 0 ? (T)0 : inverse(sum);
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        p[v] *= m.inv;
    return m;
}

// The larger of two pairs' two largest.
template <class T>
__device__ __forceinline__ void merge2(T &x, T &y, T x2, T y2)
{
    const T lo = x < x2 ? x : x2, hi = y > y2 ? y : y2;
    x = x > x2 ? x : x2;
    y = lo > hi ? lo : hi;
}

// Whether a lane's experts are all of one group, groups being `each` experts long: the
// groups' best are then found in registers.
__host__ __device__ __forceinline__ bool in_registers(int each, int vpl)
{
    const int l = each / vpl;
    return each % vpl == 0 && (l & (l - 1)) == 0;
}

// T: type of the scores, double where the keys are made of them.  LDS: a word an
// expert, and where groups need it each token's keys and its groups' (or, once the tokens
// are done, the experts' first rows).
template <int LPT, int VPL, class T>
__global__ __launch_bounds__(512) void route_kernel(const RouteArgs a)
{
    extern __shared__ __attribute__((aligned(16))) char lds[];
    const int E = a.n_experts, k = a.top_k, per = blockDim.x / LPT;
    uint64_t *const word = reinterpret_cast<uint64_t *>(lds);
    char *const own = lds + 8 * E;
    const int sub = threadIdx.x % LPT, slot = threadIdx.x / LPT, e0 = sub * VPL;
    const int each = E / a.n_groups;
    const bool groups = a.n_groups > 1, held = in_registers(each, VPL);
    T *const ks = reinterpret_cast<T *>(own) + slot * (LPT * VPL + kMaxGroups);
    const T low = -__builtin_inff();
    float b[VPL];
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        b[v] = a.bias && e0 + v < E ? a.bias[e0 + v] : 0.0f;
    for (int e = threadIdx.x; e < E; e += blockDim.x)
        word[e] = 0;
    __syncthreads();
    for (int bit = slot; bit < a.per_block; bit += per) {
        const int64_t t = (int64_t)blockIdx.x * a.per_block + bit;
        if (t >= a.tokens)
            break;
        int id = -1;
        float w = 0.0f;
        if (!(a.active && a.active[t] == 0)) {  // the same in all lanes of a token
            double key[VPL];
            Softmax<T> m;
            T x = low, y = low;  // the lane's two best, for its group
            {
                float z[VPL];
                load_logits<VPL>(a.logits, a.bf16, t * a.ldl, e0, E, z);
                T p[VPL];
                m = scores<LPT, VPL, T>(z, a.sigmoid, e0, E, p);
                if (a.bias) {
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        p[v] += (T)b[v];
                        key[v] = p[v];
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < VPL; ++v)
                        key[v] = z[v];
                }
#pragma unroll
                for (int v = 0; v < VPL; ++v)
                    key[v] = e0 + v < E ? key_of(key[v], e0 + v) : -__builtin_inf();
                // what ranks a group is made of: scores (with their bias), or logits
                if (groups && held) {
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        const T q = sizeof(T) == 8 ? p[v] : (T)z[v];
                        merge2(x, y, q == q ? q : low, low);
                    }
                } else if (groups) {
#pragma unroll
                    for (int v = 0; v < VPL; ++v) {
                        const T q = sizeof(T) == 8 ? p[v] : (T)z[v];
                        ks[e0 + v] = q == q ? q : low;
                    }
                }
            }
            if (groups && held) {
                // over the lanes of a group, then each group against the others
                const int L = each / VPL, g = sub / L, first = (threadIdx.x & 63) / LPT * LPT;
                if (L > 1)
                    merge2(x, y, other<1>(x), other<1>(y));
                if (L > 2)
                    merge2(x, y, other<2>(x), other<2>(y));
                if (L > 4)
                    merge2(x, y, other<4>(x), other<4>(y));
                if (L > 8)
                    merge2(x, y, other<8>(x), other<8>(y));
                if (L > 16)
                    merge2(x, y, other<16>(x), other<16>(y));
                x = a.two && each > 1 ? x + y : x;
                x = x == x ? x : low;
                int ahead = 0, o = g;
                for (int d = 1; d < a.n_groups; ++d) {
                    o = o + 1 == a.n_groups ? 0 : o + 1;
                    const T q = __shfl(x, first + o * L, 64);
                    ahead += q > x || (q == x && o < g) ? 1 : 0;
                }
                if (ahead >= a.top_groups) {
#pragma unroll
                    for (int v = 0; v < VPL; ++v)
                        key[v] = -__builtin_inf();
                }
            } else if (groups) {
                wave_order();
                T *const best = ks + LPT * VPL;
                for (int g = sub; g < a.n_groups; g += LPT) {
                    x = y = low;
                    for (int i = 0; i < each; ++i)
                        merge2(x, y, ks[g * each + i], low);
                    x = a.two && each > 1 ? x + y : x;
                    best[g] = x == x ? x : low;
                }
                wave_order();
                uint64_t kept = 0;
                for (int g0 = 0; g0 < a.n_groups; g0 += LPT) {
                    const int g = g0 + sub;
                    bool keep = false;
                    if (g < a.n_groups) {
                        const T mine = best[g];
                        int ahead = 0;
                        for (int i = 0; i < a.n_groups; ++i) {
                            const T q = best[i];
                            ahead += q > mine || (q == mine && i < g) ? 1 : 0;
                        }
                        keep = ahead < a.top_groups;
                    }
                    const uint64_t all = __ballot(keep);
                    const int first = (threadIdx.x & 63) / LPT * LPT;
                    const uint64_t part = LPT == 64 ? all : (all >> first) & ((1ull << (LPT & 63)) - 1);
                    kept |= part << g0;
                }
                int g = e0 / each, in = e0 - g * each;
#pragma unroll
                for (int v = 0; v < VPL; ++v) {
                    if (e0 + v < E && !(kept >> g & 1))
                        key[v] = -__builtin_inf();
                    const bool next = ++in == each;
                    g += next ? 1 : 0;
                    in = next ? 0 : in;
                }
                wave_order();  // the keys' LDS is free for the next token
            }
            sort_down(key);
            for (int j = 0; j < k; ++j) {
                const double best = max_over<LPT>(key[0]);
                id = sub == j ? expert_of(best) : id;
                if (key[0] == best) {
                    // one lane of the token steps on; a branch, as selects between
                    // neighbours of an array become a search of all of it
                    asm volatile("");
#pragma unroll
                    for (int v = 0; v + 1 < (VPL < 8 ? VPL : 8); ++v)
                        key[v] = key[v + 1];
                    if (VPL > 8 && k > 8) {
#pragma unroll
                        for (int v = 7; v + 1 < VPL; ++v)
                            key[v] = key[v + 1];
                    }
                    if (VPL <= 8 || k > 8)
                        key[VPL - 1] = -__builtin_inf();
                }
            }
            // The weight, from the logit again, as the score lies in some other lane; a sigmoid,
            // the sum and the quotient in fp32, which the result is: 6e-8 off 64 bits, of which
            // its own rounding makes 3e-8.
            if (sub < k) {
                float z[1];
                load_logits<1>(a.logits, a.bf16, t * a.ldl, id, E, z);
                w = a.sigmoid ? sigmoid_of<float>(z[0]) : (float)(m.numerator(z[0]) * m.inv);
            }
            if (a.renorm)
                w = w / (sum_over<LPT>(w) + 1e-20f);
            w *= a.scale;
        }
        if (sub < k) {
            a.weights[t * k + sub] = w;
            a.experts[t * k + sub] = id;
            if (id >= 0)
                atomicOr(reinterpret_cast<unsigned long long *>(&word[id]), 1ull << bit);
        }
    }
    __syncthreads();
    int32_t *const first = reinterpret_cast<int32_t *>(own);
    if (!a.alone) {
        for (int e = threadIdx.x; e < E; e += blockDim.x)
            a.counts[(int64_t)blockIdx.x * E + e] = __popcll(word[e]);
    } else {
        // this block is all there is: the experts' first rows
        if (threadIdx.x < 64) {
            int base = 0;
            for (int c = 0; c < E; c += 64) {
                const int e = c + threadIdx.x;
                const int n = e < E ? __popcll(word[e]) : 0;
                int sum = n;
#pragma unroll
                for (int d = 1; d < 64; d *= 2) {
                    const int o = __shfl_up(sum, d, 64);
                    sum += (int)threadIdx.x >= d ? o : 0;
                }
                if (e < E) {
                    first[e] = base + sum - n;
                    a.offsets[e] = base + sum - n;
                }
                base += __shfl(sum, 63, 64);
            }
            if (threadIdx.x == 0)
                a.offsets[E] = base;
        }
        __syncthreads();
    }
    if (sub >= k)
        return;
    for (int bit = slot; bit < a.per_block; bit += per) {
        const int64_t t = (int64_t)blockIdx.x * a.per_block + bit;
        if (t >= a.tokens)
            break;
        const int id = a.experts[t * k + sub];  // this lane's own
        a.rows_of[t * k + sub] =
            id < 0 ? -1 : __popcll(word[id] & ((1ull << bit) - 1)) + (a.alone ? first[id] : 0);
    }
}

// counts[b][e] to the sum over the blocks before b, totals[e] to the sum over all:
// 16 experts a block, 64 runs of blocks side by side.
__global__ __launch_bounds__(1024) void route_scan_kernel(int32_t *counts, int32_t *totals, int n_blocks, int E)
{
    __shared__ int32_t part[64][17];
    const int c = threadIdx.x & 15, run = threadIdx.x >> 4;
    const int e = blockIdx.x * 16 + c;
    const int per = (n_blocks + 63) / 64;
    const int b0 = run * per, b1 = b0 + per < n_blocks ? b0 + per : n_blocks;
    int s = 0;
    if (e < E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b)
            s += counts[(int64_t)b * E + e];
    }
    part[run][c] = s;
    __syncthreads();
    if (e >= E)
        return;
    int base = 0;
    for (int i = 0; i < run; ++i)
        base += part[i][c];
    if (run == 63)
        totals[e] = base + s;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
        const int64_t at = (int64_t)b * E + e;
        const int n = counts[at];
        counts[at] = base;
        base += n;
    }
}

// The same two steps in one launch, each block summing the counts for itself: 2^shift
// threads, at least E, read a row of counts, and the block's 1024 >> shift such runs of
// threads a part of the rows each.
__global__ __launch_bounds__(1024) void route_order_kernel(const int32_t *counts, const int32_t *experts,
                                                           int32_t *rows_of, int64_t *offsets, int64_t n,
                                                           int per_block, int n_blocks, int E, int shift)
{
    __shared__ int32_t all[1024], before[1024], first[kMaxExperts], wave_total[16];
    const int tid = threadIdx.x, e = tid & ((1 << shift) - 1), run = tid >> shift, runs = 1024 >> shift;
    const int per = (n_blocks + runs - 1) / runs;
    const int b0 = run * per, b1 = b0 + per < n_blocks ? b0 + per : n_blocks, mine = blockIdx.x;
    int s = 0, p = 0;
    if (e < E) {
#pragma unroll 16
        for (int b = b0; b < b1; ++b) {
            const int c = counts[(int64_t)b * E + e];
            s += c;
            p += b < mine ? c : 0;
        }
    }
    all[tid] = s;
    before[tid] = p;
    __syncthreads();
    s = p = 0;
    if (run == 0)
        for (int i = 0; i < runs; ++i) {
            s += all[(i << shift) + e];
            p += before[(i << shift) + e];
        }
    int sum = s;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(sum, d, 64);
        sum += (tid & 63) >= d ? o : 0;
    }
    if ((tid & 63) == 63)
        wave_total[tid >> 6] = sum;
    __syncthreads();
    for (int i = 0; i < tid >> 6; ++i)
        sum += wave_total[i];
    if (run == 0 && e < E) {
        first[e] = sum - s + p;
        if (mine == 0) {
            offsets[e] = sum - s;
            if (e == E - 1)
                offsets[E] = sum;
        }
    }
    __syncthreads();
    const int64_t i0 = (int64_t)mine * per_block, i1 = i0 + per_block < n ? i0 + per_block : n;
    for (int64_t i = i0 + tid; i < i1; i += 1024) {
        const int id = experts[i];
        if (id >= 0)
            rows_of[i] += first[id];
    }
}

// Adds to every choice's place in its block where its expert's rows of that block
// begin; the first block leaves the offsets.
__global__ __launch_bounds__(256) void route_place_kernel(const int32_t *counts, const int32_t *totals,
                                                          const int32_t *experts, int32_t *rows_of, int64_t *offsets,
                                                          int64_t n, int per_block, int E)
{
    __shared__ int32_t first[kMaxExperts];
    __shared__ int32_t wave_total[4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int base = 0;
    for (int c = 0; c < E; c += 256) {
        const int e = c + threadIdx.x;
        const int x = e < E ? totals[e] : 0;
        int s = x;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int o = __shfl_up(s, d, 64);
            s += lane >= d ? o : 0;
        }
        if (lane == 63)
            wave_total[w] = s;
        __syncthreads();
        int before = base;
        for (int i = 0; i < w; ++i)
            before += wave_total[i];
        base += (wave_total[0] + wave_total[1]) + (wave_total[2] + wave_total[3]);
        if (e < E) {
            first[e] = before + s - x;
            if (blockIdx.x == 0)
                offsets[e] = before + s - x;
        }
        __syncthreads();
    }
    if (blockIdx.x == 0 && threadIdx.x == 0)
        offsets[E] = base;
    const int64_t i0 = (int64_t)blockIdx.x * per_block;
    const int64_t i1 = i0 + per_block < n ? i0 + per_block : n;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += 256) {
        const int e = experts[i];
        if (e >= 0)
            rows_of[i] += first[e] + counts[(int64_t)blockIdx.x * E + e];
    }
}

struct RouteBackArgs {
    int64_t tokens, ldl, ldd;
    const void *logits;
    const int32_t *experts;
    const float *dweights;
    void *dlogits;
    float scale;
    int32_t n_experts, top_k;
    bool sigmoid, renorm, l_bf16, d_bf16;
};

// With w_j = scale s_j (/ S, S = sum of the chosen s + 1e-20) and D = dw scale:
//   ds_j = D_j, or (D_j - sum D s / S) / S;
//   softmax: dl_i = s_i (ds_i - sum ds s);  sigmoid: dl_i = ds_i s_i (1 - s_i).
// The scores come again from the logits.  A token's ds lie in LDS, scattered by
// its experts' numbers.
template <int LPT, int VPL>
__global__ __launch_bounds__(256) void route_backward_kernel(const RouteBackArgs a)
{
    constexpr int TPB = 256 / LPT;
    __shared__ float scatter[TPB][LPT * VPL];
    const int E = a.n_experts, k = a.top_k;
    const int sub = threadIdx.x % LPT, slot = threadIdx.x / LPT, e0 = sub * VPL;
    const int64_t t = (int64_t)blockIdx.x * TPB + slot;
    if (t >= a.tokens)
        return;
    float *const ds = scatter[slot];
    float z[VPL], p[VPL];
    load_logits<VPL>(a.logits, a.l_bf16, t * a.ldl, e0, E, z);
    const int id = sub < k ? a.experts[t * k + sub] : -1;
    const bool chosen = id >= 0 && id < E;
    float d = chosen ? a.dweights[t * k + sub] * a.scale : 0.0f;
    scores<LPT, VPL, float>(z, a.sigmoid, e0, E, p);
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        ds[e0 + v] = p[v];
    wave_order();
    const float s = chosen ? ds[id] : 0.0f;
    const int n_chosen = sum_over<LPT>(chosen ? 1 : 0);
    if (a.renorm) {
        const float total = sum_over<LPT>(s) + 1e-20f;
        const float mean = sum_over<LPT>(d * s) / total;
        // of one expert alone d - mean is d 1e-20 / total, which the difference loses
        d = !chosen ? 0.0f : n_chosen == 1 ? d * (1e-20f / total) / total : (d - mean) / total;
    }
    const float dot = sum_over<LPT>(d * s);
    wave_order();
#pragma unroll
    for (int v = 0; v < VPL; ++v)
        ds[e0 + v] = 0.0f;
    wave_order();
    if (chosen)
        atomicAdd(&ds[id], d);  // of one token's experts no two are the same
    wave_order();
    float dz[VPL];  // 0 for a token without experts
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
        const float x = ds[e0 + v];
        // 1 - s is e^-z s where s is the larger: the difference would lose all of it past z = 17
        const float rest = z[v] > 0.0f ? exp_below(-z[v]) * p[v] : 1.0f - p[v];
        dz[v] = n_chosen == 0 ? 0.0f : a.sigmoid ? x * (p[v] * rest) : p[v] * (x - dot);
    }
    const int64_t at = t * a.ldd;
    if constexpr (VPL >= 8) {
#pragma unroll
        for (int v = 0; v < VPL; v += 8) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[i] = dz[v + i];
            const int n = E - e0 - v < 8 ? E - e0 - v : 8;
            if (n > 0)
                store8(a.dlogits, a.d_bf16, at + e0 + v, n == 8, n, w);
        }
    } else {
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
            if (e0 + v >= E)
                continue;
            if (a.d_bf16)
                static_cast<uint16_t *>(a.dlogits)[at + e0 + v] = (uint16_t)pack_bf16(dz[v], dz[v]);
            else
                static_cast<float *>(a.dlogits)[at + e0 + v] = dz[v];
        }
    }
}

// ----------------------------------------------------------- the moves --

struct MoveArgs {
    int64_t tokens, cols, rows;
    const uint16_t *x;  // tokens x cols
    const uint16_t *e;  // rows x cols, sorted
    uint16_t *out;      // rows x cols, sorted
    void *y;            // tokens x cols
    const uint16_t *residual;
    const int32_t *rows_of;
    const float *weights;
    float *dweights;
    int64_t ldx, lde, ldo, ldy, ldr;
    int32_t top_k, shift;  // 1 << shift lanes a token
    bool y_bf16;
};

// Row of choice j of token t, -1 where it is none of the `rows`.
__device__ __forceinline__ int64_t row_at(const MoveArgs &a, int64_t t, int j)
{
    const int64_t r = a.rows_of[t * a.top_k + j];
    return r >= 0 && r < a.rows ? r : -1;
}

// out[row] = w x[t] for each of token t's rows.
__global__ __launch_bounds__(256) void dispatch_kernel(const MoveArgs a)
{
    const int lanes = 1 << a.shift;
    const int64_t t = ((int64_t)blockIdx.x << (8 - a.shift)) + (threadIdx.x >> a.shift);
    if (t >= a.tokens)
        return;
    for (int64_t c = (threadIdx.x & (lanes - 1)) * 8; c < a.cols; c += 8 * lanes) {
        const int n = (int)(a.cols - c < 8 ? a.cols - c : 8);
        float x[8], y[8];
        load8(a.x, true, t * a.ldx + c, n == 8, n, x);
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t r = row_at(a, t, j);
            if (r < 0)
                continue;
            const float w = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = a.weights ? x[i] * w : x[i];
            store8(a.out, true, r * a.ldo + c, n == 8, n, y);
        }
    }
}

// y[t] = sum over j of w e[row] (+ residual), in order of j.
__global__ __launch_bounds__(256) void combine_kernel(const MoveArgs a)
{
    const int lanes = 1 << a.shift;
    const int64_t t = ((int64_t)blockIdx.x << (8 - a.shift)) + (threadIdx.x >> a.shift);
    if (t >= a.tokens)
        return;
    for (int64_t c = (threadIdx.x & (lanes - 1)) * 8; c < a.cols; c += 8 * lanes) {
        const int n = (int)(a.cols - c < 8 ? a.cols - c : 8);
        float s[8] = {};
#pragma unroll 4
        for (int j = 0; j < a.top_k; ++j) {
            const int64_t r = row_at(a, t, j);
            if (r < 0)
                continue;
            const float w = a.weights ? a.weights[t * a.top_k + j] : 1.0f;
            float x[8];
            load8(a.e, true, r * a.lde + c, n == 8, n, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] = __builtin_fmaf(w, x[i], s[i]);
        }
        if (a.residual) {
            float x[8];
            load8(a.residual, true, t * a.ldr + c, n == 8, n, x);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                s[i] += x[i];
        }
        store8(a.y, a.y_bf16, t * a.ldy + c, n == 8, n, s);
    }
}

// out[row] = w dy[t], dw[t][j] = sum over the columns of dy[t] e[row].
template <int K>
__global__ __launch_bounds__(256) void combine_backward_kernel(const MoveArgs a)
{
    __shared__ float part[4][K];
    const int lanes = 1 << a.shift;
    const int64_t t = ((int64_t)blockIdx.x << (8 - a.shift)) + (threadIdx.x >> a.shift);
    const int lane = threadIdx.x & (lanes - 1);
    const bool here = t < a.tokens;
    float dot[K];
    int64_t row[K];
    float w[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        dot[j] = 0.0f;
        row[j] = -1;
        w[j] = 0.0f;
    }
    if (here && a.cols > 0) {
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (j < a.top_k) {
                row[j] = row_at(a, t, j);
                w[j] = a.weights[t * a.top_k + j];
            }
    }
    for (int64_t c = (int64_t)lane * 8; here && c < a.cols; c += 8 * lanes) {
        const int n = (int)(a.cols - c < 8 ? a.cols - c : 8);
        float dy[8], d[8];
        load8(a.x, true, t * a.ldx + c, n == 8, n, dy);
        auto one = [&](int j, const float (&e)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dot[j] = __builtin_fmaf(dy[i], e[i], dot[j]);
                d[i] = w[j] * dy[i];
            }
            store8(a.out, true, row[j] * a.ldo + c, n == 8, n, d);
        };
        if (n == 8) {
            // every row's load before the first store, which could be to a row; none's
            // is one of dy, which is there, so that no branch parts the loads
            uint4 raw[K];
#pragma unroll
            for (int j = 0; j < K; ++j)
                raw[j] = load16(row[j] < 0 ? a.x + t * a.ldx + c : a.e + row[j] * a.lde + c);
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float e[8];
                widen8(raw[j], e);
                if (row[j] >= 0)
                    one(j, e);
            }
        } else {
#pragma unroll
            for (int j = 0; j < K; ++j) {
                float e[8];
                if (row[j] < 0)
                    continue;
                load8(a.e, true, row[j] * a.lde + c, false, n, e);
                one(j, e);
            }
        }
    }
    // lanes of one token: part of a wave, or the whole block
#pragma unroll
    for (int j = 0; j < K; ++j)
        for (int s = 1; s < lanes && s < 64; s *= 2)
            dot[j] += __shfl_xor(dot[j], s, 64);
    if (lanes > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int j = 0; j < K; ++j)
                part[threadIdx.x >> 6][j] = dot[j];
        __syncthreads();
        const int w0 = (threadIdx.x >> a.shift) << (a.shift - 6);
#pragma unroll
        for (int j = 0; j < K; ++j) {
            dot[j] = part[w0][j];
            for (int i = 1; i < lanes / 64; ++i)
                dot[j] += part[w0 + i][j];
        }
    }
    if (here && lane == 0)
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (j < a.top_k)
                a.dweights[t * a.top_k + j] = dot[j];
}

// ---------------------------------------------------------------- host --

zero_status check_router(const zero_router *r)
{
    if (!r)
        return fail(ZERO_ERR_INVALID_ARG, "the router is NULL");
    if (r->n_experts < 1 || r->top_k < 1 || r->n_groups < 1 || r->top_groups < 1)
        return fail(ZERO_ERR_INVALID_ARG, "a router needs experts, top_k, groups and top_groups of at least 1");
    if (r->n_experts > kMaxExperts || r->top_k > kMaxTopK || r->n_groups > kMaxGroups)
        return fail(ZERO_ERR_UNSUPPORTED, "at most %d experts, %d of them for a token, and %d groups", kMaxExperts,
                    kMaxTopK, kMaxGroups);
    if (r->n_experts % r->n_groups || r->top_groups > r->n_groups)
        return fail(ZERO_ERR_INVALID_ARG, "%d groups (%d kept) of %d experts", r->n_groups, r->top_groups,
                    r->n_experts);
    if (r->top_k > r->top_groups * (r->n_experts / r->n_groups))
        return fail(ZERO_ERR_INVALID_ARG, "top_k %d is more than the kept groups have", r->top_k);
    if (r->group_best != 1 && r->group_best != 2)
        return fail(ZERO_ERR_INVALID_ARG, "group_best must be 1 or 2");
    if (r->score != ZERO_SCORE_SOFTMAX && r->score != ZERO_SCORE_SIGMOID)
        return fail(ZERO_ERR_INVALID_ARG, "unknown score %d", r->score);
    if (!(r->scale - r->scale == 0.0f))
        return fail(ZERO_ERR_INVALID_ARG, "scale must be finite");
    return ZERO_OK;
}

zero_status check_tokens(int64_t tokens, int32_t top_k)
{
    if (tokens < 0)
        return fail(ZERO_ERR_INVALID_ARG, "negative number of tokens");
    if (tokens > int64_t(0x7fffffff) / top_k)
        return fail(ZERO_ERR_UNSUPPORTED, "tokens x top_k must fit 31 bits");
    return ZERO_OK;
}

// Lanes a token and experts a lane for E experts: at most MOST a lane while there are
// lanes.
template <int MOST = 16, class F>
void by_experts(int E, F f)
{
#define ZS_CASE(L, V) f(std::integral_constant<int, L>{}, std::integral_constant<int, V>{})
    if (E <= 16)
        ZS_CASE(16, 1);
    else if (E <= 32)
        ZS_CASE(16, 2);
    else if (E <= 64)
        ZS_CASE(16, 4);
    else if (E <= 128)
        ZS_CASE(128 / (MOST < 8 ? MOST : 8), (MOST < 8 ? MOST : 8));
    else if (E <= 256)
        ZS_CASE(256 / MOST, MOST);
    else if (E <= 512)
        ZS_CASE((MOST < 8 ? 64 : 512 / MOST), (MOST < 8 ? 8 : MOST));
    else
        ZS_CASE(64, 16);
#undef ZS_CASE
}

// Whether a router's groups need LDS for every key.
bool group_keys(const zero_router *r)
{
    bool keys = false;
    if (r->n_groups > 1)
        by_experts(r->n_experts, [&](auto, auto vc) {
            keys = !in_registers(r->n_experts / r->n_groups, decltype(vc)::value);
        });
    return keys;
}

int route_per_block(const zero_router *r) { return group_keys(r) ? kGroupTokens : kRouteTokens; }
// Threads of a full block: with groups' keys, of at most 43 KB, 256.
int route_threads(const zero_router *r) { return group_keys(r) ? 256 : 512; }
int64_t route_blocks(const zero_router *r, int64_t tokens)
{
    const int n = route_per_block(r);
    return (tokens + n - 1) / n;
}

// Lanes a token, as a power of two: 8 columns each, a block at most.
int lanes_shift(int64_t cols)
{
    int s = 0;
    while (s < 8 && (int64_t(8) << s) < cols)
        ++s;
    return s;
}

zero_status check_move(int64_t tokens, int32_t top_k, int64_t cols, int64_t rows, const int32_t *rows_of,
                       const float *weights)
{
    zero_status st;
    if (top_k < 1)
        return fail(ZERO_ERR_INVALID_ARG, "top_k must be at least 1");
    if (top_k > kMaxTopK)
        return fail(ZERO_ERR_UNSUPPORTED, "top_k is at most %d", kMaxTopK);
    if ((st = check_tokens(tokens, top_k)) != ZERO_OK || (st = check_extent(rows, cols, cols)) != ZERO_OK)
        return st;
    if (tokens == 0 || cols == 0)
        return ZERO_OK;
    if (!rows_of)
        return fail(ZERO_ERR_INVALID_ARG, "rows_of is required");
    if (!aligned(rows_of, 4) || !aligned(weights, 4))
        return fail(ZERO_ERR_ALIGNMENT, "rows_of and weights must be 4-byte aligned");
    return ZERO_OK;
}

zero_status check_side(const char *what, const void *p, int64_t ld, int64_t rows, int64_t cols, int32_t dtype)
{
    const zero_status st = check_extent(rows, cols, ld);
    if (st != ZERO_OK || rows == 0)
        return st;
    return check_matrix(what, p, ld, cols, dtype);
}

// The dispatch counts a launch's threads in 32 bits.
constexpr int64_t kMaxThreads = 0xffffffffu;

// go(args, blocks) for all tokens, as many at a time as a launch has blocks for.
template <class F>
zero_status each_launch(MoveArgs a, const char *what, F go)
{
    const int64_t per = 256 >> a.shift, most = kMaxThreads / 256 * per;
    const int64_t es = a.y_bf16 ? 2 : 4;
    (void)hipGetLastError();
    for (int64_t left = a.tokens; left > 0; left -= most) {
        a.tokens = left < most ? left : most;
        go(a, dim3((unsigned)((a.tokens + per - 1) / per)));
        const zero_status st = launched(what);
        if (st != ZERO_OK || left <= most)
            return st;
        a.rows_of += most * a.top_k;
        if (a.x)
            a.x += most * a.ldx;
        if (a.y)
            a.y = static_cast<char *>(a.y) + most * a.ldy * es;
        if (a.residual)
            a.residual += most * a.ldr;
        if (a.weights)
            a.weights += most * a.top_k;
        if (a.dweights)
            a.dweights += most * a.top_k;
    }
    return ZERO_OK;
}

}  // namespace
}  // namespace zs

extern "C" {

int64_t zero_route_workspace(const zero_router *r, int64_t tokens)
{
    if (!r || r->n_experts < 1 || tokens < 0)
        return 0;
    const int64_t b = zs::route_blocks(r, tokens);
    return b > 1 ? (b + 1) * r->n_experts : 0;
}

zero_status zero_route_forward(const zero_router *r, int64_t tokens, const void *logits, int64_t ldl,
                               int32_t logits_dtype, const float *bias, const uint8_t *active, int32_t *experts,
                               float *weights, int64_t *offsets, int32_t *rows_of, int32_t *workspace,
                               int64_t n_workspace, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_router(r)) != ZERO_OK || (st = check_tokens(tokens, r->top_k)) != ZERO_OK ||
        (st = check_extent(tokens, r->n_experts, ldl)) != ZERO_OK)
        return st;
    if (!known_dtype(logits_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "logits: unknown dtype %d", logits_dtype);
    if (!offsets || (tokens > 0 && (!experts || !weights || !rows_of)))
        return fail(ZERO_ERR_INVALID_ARG, "experts, weights, offsets and rows_of are required");
    if (tokens > 0 && (st = check_matrix("logits", logits, ldl, r->n_experts, logits_dtype)) != ZERO_OK)
        return st;
    if (!aligned(offsets, 8) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(rows_of, 4) ||
        !aligned(bias, 4) || !aligned(workspace, 4))
        return fail(ZERO_ERR_ALIGNMENT, "a routing buffer is misaligned");
    if (route_blocks(r, tokens) > kMaxThreads / route_threads(r))
        return fail(ZERO_ERR_UNSUPPORTED, "%lld tokens are too many for one launch", (long long)tokens);
    const int64_t need = zero_route_workspace(r, tokens);
    if (need > 0 && (!workspace || n_workspace < need))
        return fail(ZERO_ERR_INVALID_ARG, "routing %lld tokens needs a workspace of %lld int32", (long long)tokens,
                    (long long)need);
    const void *w = need > 0 ? workspace : nullptr, *l = tokens > 0 ? logits : nullptr;
    if (is_one_of(experts, {weights, offsets, rows_of, w, l, bias, active}) ||
        is_one_of(weights, {offsets, rows_of, w, l, bias, active}) ||
        is_one_of(offsets, {rows_of, w, l, bias, active}) || is_one_of(rows_of, {w, l, bias, active}) ||
        is_one_of(w, {l, bias, active}))
        return fail(ZERO_ERR_INVALID_ARG, "each result and the workspace need memory of their own");
    RouteArgs a = {};
    a.tokens = tokens, a.ldl = ldl, a.logits = logits, a.bias = bias, a.active = active;
    a.experts = experts, a.weights = weights, a.offsets = offsets, a.rows_of = rows_of;
    a.n_experts = r->n_experts, a.top_k = r->top_k, a.n_groups = r->n_groups, a.top_groups = r->top_groups;
    a.scale = r->scale, a.sigmoid = r->score == ZERO_SCORE_SIGMOID, a.renorm = r->renormalize != 0;
    a.two = r->group_best == 2, a.bf16 = logits_dtype == ZERO_BF16;
    const int64_t blocks = tokens > 0 ? route_blocks(r, tokens) : 1;
    a.per_block = route_per_block(r);
    a.alone = blocks == 1;
    a.counts = workspace;
    a.totals = workspace ? workspace + blocks * r->n_experts : nullptr;
    const int E = r->n_experts;
    // keys that are sums of scores need fp64
    const bool deep = bias || (r->n_groups > 1 && a.two);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    by_experts(E, [&](auto lc, auto vc) {
        constexpr int LPT = decltype(lc)::value, VPL = decltype(vc)::value;
        // as many threads as the block's tokens keep busy
        const int64_t most = tokens < a.per_block ? tokens : a.per_block;
        const int limit = route_threads(r);
        int threads = 64;
        while (threads < limit && threads / LPT < most)
            threads *= 2;
        const int own = group_keys(r) ? threads / LPT * (LPT * VPL + kMaxGroups) * (deep ? 8 : 4) : 0;
        const size_t lds = 8 * (size_t)E + (size_t)(own > 4 * E ? own : 4 * E);
        if (deep)
            hipLaunchKernelGGL((route_kernel<LPT, VPL, double>), dim3((unsigned)blocks), dim3(threads), lds, s, a);
        else
            hipLaunchKernelGGL((route_kernel<LPT, VPL, float>), dim3((unsigned)blocks), dim3(threads), lds, s, a);
    });
    if ((st = launched("route")) != ZERO_OK || a.alone)
        return st;
    int shift = 6;
    while ((1 << shift) < E)
        ++shift;
    // One launch or two, us in all: 200 tokens of 64 10.4 and 12.8, 16384 of 64 12.4 and
    // 15.3, 8192 of 256 19.8 and 21.0; 16384 of 256 23.2 and 23.5, 8192 of 512 35.2 and
    // 34.9, 32768 of 64 18.4 and 17.5.  So one up to 32 counts a thread.
    if (blocks << shift <= 32768) {
        hipLaunchKernelGGL(route_order_kernel, dim3((unsigned)blocks), dim3(1024), 0, s, a.counts, experts, rows_of,
                           offsets, tokens * r->top_k, a.per_block * r->top_k, (int)blocks, E, shift);
        return launched("route order");
    }
    hipLaunchKernelGGL(route_scan_kernel, dim3((unsigned)((E + 15) / 16)), dim3(1024), 0, s, a.counts, a.totals,
                       (int)blocks, E);
    hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a.counts, a.totals, experts, rows_of,
                       offsets, tokens * r->top_k, a.per_block * r->top_k, E);
    return launched("route order");
}

zero_status zero_route_backward(const zero_router *r, int64_t tokens, const void *logits, int64_t ldl,
                                int32_t logits_dtype, const int32_t *experts, const float *dweights, void *dlogits,
                                int64_t ldd, int32_t dlogits_dtype, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_router(r)) != ZERO_OK || (st = check_tokens(tokens, r->top_k)) != ZERO_OK ||
        (st = check_extent(tokens, r->n_experts, ldl)) != ZERO_OK ||
        (st = check_extent(tokens, r->n_experts, ldd)) != ZERO_OK)
        return st;
    if (!known_dtype(logits_dtype) || !known_dtype(dlogits_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "unknown dtype (logits %d, dlogits %d)", logits_dtype, dlogits_dtype);
    if (tokens == 0)
        return ZERO_OK;
    if ((st = check_matrix("logits", logits, ldl, r->n_experts, logits_dtype)) != ZERO_OK ||
        (st = check_matrix("dlogits", dlogits, ldd, r->n_experts, dlogits_dtype)) != ZERO_OK)
        return st;
    if (!experts || !dweights)
        return fail(ZERO_ERR_INVALID_ARG, "experts and dweights are required");
    if (!aligned(experts, 4) || !aligned(dweights, 4))
        return fail(ZERO_ERR_ALIGNMENT, "experts and dweights must be 4-byte aligned");
    if (dlogits == logits && (ldd != ldl || dlogits_dtype != logits_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "dlogits in place of logits needs their type and leading dimension");
    if (is_one_of(dlogits, {experts, dweights}))
        return fail(ZERO_ERR_INVALID_ARG, "dlogits needs memory apart from what the call reads");
    RouteBackArgs a = {};
    a.tokens = tokens, a.ldl = ldl, a.ldd = ldd, a.logits = logits, a.experts = experts, a.dweights = dweights;
    a.dlogits = dlogits, a.scale = r->scale, a.n_experts = r->n_experts, a.top_k = r->top_k;
    a.sigmoid = r->score == ZERO_SCORE_SIGMOID, a.renorm = r->renormalize != 0;
    a.l_bf16 = logits_dtype == ZERO_BF16, a.d_bf16 = dlogits_dtype == ZERO_BF16;
    (void)hipGetLastError();
    by_experts<8>(r->n_experts, [&](auto lc, auto vc) {
        constexpr int LPT = decltype(lc)::value, VPL = decltype(vc)::value, TPB = 256 / LPT;
        // as many tokens at a time as a launch has blocks for
        constexpr int64_t most = kMaxThreads / 256 * TPB;
        for (int64_t t0 = 0; t0 < tokens && st == ZERO_OK; t0 += most) {
            a.tokens = tokens - t0 < most ? tokens - t0 : most;
            a.logits = static_cast<const char *>(logits) + t0 * ldl * bytes_of(logits_dtype);
            a.dlogits = static_cast<char *>(dlogits) + t0 * ldd * bytes_of(dlogits_dtype);
            a.experts = experts + t0 * a.top_k;
            a.dweights = dweights + t0 * a.top_k;
            hipLaunchKernelGGL((route_backward_kernel<LPT, VPL>), dim3((unsigned)((a.tokens + TPB - 1) / TPB)),
                               dim3(256), 0, static_cast<hipStream_t>(stream), a);
            st = launched("route_backward");
        }
    });
    return st;
}

zero_status zero_experts_dispatch(int64_t tokens, int32_t top_k, int64_t cols, const uint16_t *x, int64_t ldx,
                                  const int32_t *rows_of, const float *weights, int64_t rows, uint16_t *out,
                                  int64_t ldo, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_move(tokens, top_k, cols, rows, rows_of, weights)) != ZERO_OK)
        return st;
    if (tokens == 0 || cols == 0)
        return ZERO_OK;
    if ((st = check_side("x", x, ldx, tokens, cols, ZERO_BF16)) != ZERO_OK ||
        (st = check_side("out", out, ldo, rows, cols, ZERO_BF16)) != ZERO_OK)
        return st;
    if (rows == 0)
        return ZERO_OK;
    if (is_one_of(out, {x, rows_of, weights}))
        return fail(ZERO_ERR_INVALID_ARG, "the moved rows need memory apart from what the call reads");
    MoveArgs a = {};
    a.tokens = tokens, a.cols = cols, a.rows = rows, a.x = x, a.ldx = ldx, a.out = out, a.ldo = ldo;
    a.rows_of = rows_of, a.weights = weights, a.top_k = top_k, a.shift = lanes_shift(cols);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return each_launch(a, "experts_dispatch", [&](const MoveArgs &m, dim3 grid) {
        hipLaunchKernelGGL(dispatch_kernel, grid, dim3(256), 0, s, m);
    });
}

zero_status zero_experts_combine(int64_t tokens, int32_t top_k, int64_t cols, const uint16_t *in, int64_t ldi,
                                 int64_t rows, const int32_t *rows_of, const float *weights,
                                 const uint16_t *residual, int64_t ldr, void *y, int64_t ldy, int32_t y_dtype,
                                 void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_move(tokens, top_k, cols, rows, rows_of, weights)) != ZERO_OK)
        return st;
    if (!known_dtype(y_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "y: unknown dtype %d", y_dtype);
    if (tokens == 0 || cols == 0)
        return ZERO_OK;
    if ((st = check_side("in", in, ldi, rows, cols, ZERO_BF16)) != ZERO_OK ||
        (st = check_side("y", y, ldy, tokens, cols, y_dtype)) != ZERO_OK ||
        (residual && (st = check_side("residual", residual, ldr, tokens, cols, ZERO_BF16)) != ZERO_OK))
        return st;
    if (y == residual && (y_dtype != ZERO_BF16 || ldy != ldr))
        return fail(ZERO_ERR_INVALID_ARG, "y in place of the residual needs bf16 and the same leading dimension");
    if (is_one_of(y, {rows > 0 ? in : nullptr, rows_of, weights}))
        return fail(ZERO_ERR_INVALID_ARG, "y needs memory apart from what the call reads");
    MoveArgs a = {};
    a.tokens = tokens, a.cols = cols, a.rows = rows, a.e = in, a.lde = ldi, a.y = y, a.ldy = ldy;
    a.rows_of = rows_of, a.weights = weights, a.top_k = top_k, a.shift = lanes_shift(cols);
    a.residual = residual, a.ldr = ldr, a.y_bf16 = y_dtype == ZERO_BF16;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return each_launch(a, "experts_combine", [&](const MoveArgs &m, dim3 grid) {
        hipLaunchKernelGGL(combine_kernel, grid, dim3(256), 0, s, m);
    });
}

zero_status zero_experts_combine_backward(int64_t tokens, int32_t top_k, int64_t cols, const uint16_t *dy,
                                          int64_t lddy, int64_t rows, const int32_t *rows_of, const float *weights,
                                          const uint16_t *in, int64_t ldi, uint16_t *din, int64_t lddi,
                                          float *dweights, void *stream)
{
    using namespace zs;
    zero_status st;
    if ((st = check_move(tokens, top_k, cols, rows, rows_of, weights)) != ZERO_OK)
        return st;
    if (tokens == 0)
        return ZERO_OK;
    if (!dweights || !aligned(dweights, 4))
        return fail(dweights ? ZERO_ERR_ALIGNMENT : ZERO_ERR_INVALID_ARG, "dweights is required, 4-byte aligned");
    if (cols > 0) {
        if (!weights)
            return fail(ZERO_ERR_INVALID_ARG, "weights are required");
        if ((st = check_side("dy", dy, lddy, tokens, cols, ZERO_BF16)) != ZERO_OK ||
            (st = check_side("in", in, ldi, rows, cols, ZERO_BF16)) != ZERO_OK ||
            (st = check_side("din", din, lddi, rows, cols, ZERO_BF16)) != ZERO_OK)
            return st;
        if (rows > 0 && din == in && lddi != ldi)
            return fail(ZERO_ERR_INVALID_ARG, "din in place of in needs the same leading dimension");
        const void *e = rows > 0 ? in : nullptr, *d = rows > 0 ? din : nullptr;
        if (is_one_of(d, {dy, rows_of, weights, dweights}) || is_one_of(dweights, {dy, rows_of, weights, e}))
            return fail(ZERO_ERR_INVALID_ARG, "din and dweights need memory apart from what the call reads and from "
                        "each other");
    }
    MoveArgs a = {};
    a.tokens = tokens, a.cols = cols, a.rows = rows, a.x = dy, a.ldx = lddy, a.e = in, a.lde = ldi, a.out = din;
    a.ldo = lddi, a.rows_of = rows_of, a.weights = weights, a.dweights = dweights, a.top_k = top_k;
    a.shift = lanes_shift(cols);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return each_launch(a, "experts_combine_backward", [&](const MoveArgs &m, dim3 grid) {
        if (top_k <= 1)
            hipLaunchKernelGGL(combine_backward_kernel<1>, grid, dim3(256), 0, s, m);
        else if (top_k <= 2)
            hipLaunchKernelGGL(combine_backward_kernel<2>, grid, dim3(256), 0, s, m);
        else if (top_k <= 4)
            hipLaunchKernelGGL(combine_backward_kernel<4>, grid, dim3(256), 0, s, m);
        else if (top_k <= 8)
            hipLaunchKernelGGL(combine_backward_kernel<8>, grid, dim3(256), 0, s, m);
        else
            hipLaunchKernelGGL(combine_backward_kernel<16>, grid, dim3(256), 0, s, m);
    });
}

}  // extern "C"
