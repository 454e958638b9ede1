// Adam / AdamW over many tensors at once, with fp32 states or states in 8 bits,
// and what belongs to it: the sum of squares of the tensors' gradients (for a
// global-norm clip) and the values of 8-bit states.
//
// A launch takes up to kTensors tensors from its arguments and walks their
// concatenated tiles of 2048 elements, a lane eight neighbouring ones, so that
// many small tensors cost one launch between them.  An element costs 2 or 4
// bytes of gradient, 8 of master, 2 of parameter and 16 (fp32) or 4 1/8 bytes of
// state, and no product: memory bounds it.  267 M elements in 180 tensors with bf16
// gradients: 8-bit states 0.78 to 0.82 ms in four launches, 5.3 to 5.6 TB/s; fp32 states
// 1.39 ms, 5.4 TB/s; where a copy of 4 GB reaches 6.6.  The sums of squares of those
// gradients take 107 us, 5.0 TB/s (fp32 ones 179, 6.0).
//
// 8-bit states.  m and the root of v are kept as e4m3 codes, 32 neighbouring
// elements of a tensor under one power of two: the least 2^e, e in [-117, 120],
// with the block's largest finite magnitude at most 448 * 2^e.  The root halves
// v's range of exponents, so that a block whose gradients span five decades
// still has a code for each.  The codes' step is 1/16 to 1/8 of a value and an
// exponential average moves v by (1 - beta2) of itself a step, so rounding to
// nearest would leave v where it is for good; a new state is therefore rounded
// up or down at random, up with the probability of the part that rounding down
// would lose, which keeps the average right.  A v that is not 0 keeps a code
// that is not 0: it would else be missing under a later m.  The step itself uses
// m and v before they are rounded.
//
// The random bits are a hash of the element's number in the list, the seed and
// the step number, so a step has the same bits whatever the launch, and needs no
// state of its own.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstddef>
#include <cstring>

#include "act.h"
#include "checks.h"
#include "vec.h"
#include "zero_shard.h"

#pragma clang fp contract(off)

namespace zs {
namespace {

// The step scalars; the same layout as zero_adam_table_entry, so a table of
// them in device memory can be read as is.
struct AdamScalars {
    float lr, b1, b2, eps, wd;
    float omb1, omb2, bias1, bias2, decay;
    int32_t has_wd, decoupled;
};
static_assert(sizeof(AdamScalars) == sizeof(zero_adam_table_entry), "table entry layout");
static_assert(offsetof(AdamScalars, omb1) == offsetof(zero_adam_table_entry, one_minus_beta1) &&
                  offsetof(AdamScalars, decay) == offsetof(zero_adam_table_entry, decay) &&
                  offsetof(AdamScalars, has_wd) == offsetof(zero_adam_table_entry, has_decay) &&
                  offsetof(AdamScalars, decoupled) == offsetof(zero_adam_table_entry, decoupled),
              "table entry layout");

// The shard step's arithmetic (kernels.hip), operation by operation, so that a tensor with
// fp32 states gets the bits it would get there.
__device__ __forceinline__ void adam1(const AdamScalars &s, float g, float &p, float &m, float &v)
{
    if (s.has_wd) {
        if (s.decoupled)
            p = p * s.decay;
        else
            g = g + s.wd * p;
    }
    m = s.b1 * m + s.omb1 * g;
    v = s.b2 * v + s.omb2 * (g * g);
    const float m_hat = m / s.bias1;
    const float v_hat = v / s.bias2;
    const float denom = sqrtf(v_hat) + s.eps;
    p = p - s.lr * (m_hat / denom);
}

constexpr int kTensors = 50;     // tensors of one launch, at most a wave's lanes: its arguments stay below 4 KB
constexpr int kTensorTile = 2048;
constexpr int kSumTile = 8192;   // elements of one sum of squares

struct Tensor {
    float *master;
    const void *grad;
    uint16_t *param;
    void *m, *v;
    uint8_t *ms, *vs;
    int64_t n, number;  // elements, the first one's number in the list
};

struct TensorArgs {
    AdamScalars sc;
    float rate, per;           // 8-bit states: lr / bias1, 1 / sqrt(bias2)
    const AdamScalars *table;  // non-null: scalars of table[*counter - 1]
    const int64_t *counter;
    int64_t n_table, step, first_sum;
    uint64_t seed;
    const float *clip;
    double *sums;
    uint64_t decay;            // a bit a tensor
    int32_t n_tensors, g_bf16;
    int32_t tile0[kTensors];   // each tensor's first tile
    Tensor t[kTensors];
};
static_assert(sizeof(TensorArgs) <= 4096, "kernel arguments");

// The tensor that a tile belongs to: a lane looks at one tensor each (a search in steps
// waits for each of its reads: 12 small tensors 8.3 us, so 7.7).
__device__ __forceinline__ int tensor_of(const TensorArgs &a, int tile)
{
    const int lane = threadIdx.x & 63;
    const int first = a.tile0[lane < a.n_tensors ? lane : 0];
    return __popcll(__ballot(lane < a.n_tensors && first <= tile)) - 1;
}

// The step's two keys: rounds of xor-shift and multiplication over the seed and the step
// number, which enters by multiples of the golden ratio's fraction of 2^64.  Here and
// below a multiplier has to be odd, so that a round loses nothing, and to hold about as
// many ones as zeros in no pattern, so that a bit reaches all above it; nothing else
// hangs on its value.
__device__ __forceinline__ uint2 step_keys(uint64_t seed, int64_t step)
{
    uint64_t z = seed + (uint64_t)step * 0x9E3779B97F4A7C15ull;
    z = (z ^ (z >> 31)) * 0xD6E8FEB86659FD93ull;
    z = (z ^ (z >> 29)) * 0xA0761D6478BD642Full;
    z ^= z >> 32;
    return make_uint2((uint32_t)z, (uint32_t)(z >> 32));
}

// 32 random bits of element number i.
__device__ __forceinline__ uint32_t random_bits(uint2 key, int64_t i)
{
    uint32_t h = (uint32_t)i * 0x9E3779B1u + (uint32_t)((uint64_t)i >> 32) * 0x85EBCA77u + key.x;
    h ^= h >> 16;
    h = h * 0x7FEB352Du + key.y;
    h ^= h >> 15;
    h *= 0x6C8E9CF5u;
    return h ^ (h >> 16);
}

template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t x)
{
    const uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, true);
    return x > y ? x : y;
}

// Largest of the four lanes of a block of 32.
__device__ __forceinline__ uint32_t over_block(uint32_t mx)
{
    mx = quad_max<0xB1>(mx);  // lanes 1 0 3 2
    return quad_max<0x4E>(mx);  // lanes 2 3 0 1
}

constexpr uint32_t kLimBits = 0x7f700000u;  // 240 * 2^120

// x / 2^e as a code (ROOT: x is not negative), rounded up where the 16 random bits
// `r` and the part of a step above the code below sum to a whole step.  Under 2^-6
// the codes are 2^-9 apart, as they are from 2^-6 to 2^-5, so 2^-6 is added there.
// PLAIN: x is finite and at most 240 * 2^120.
template <bool ROOT, bool PLAIN>
__device__ __forceinline__ uint32_t code_random(float x, float inv, uint32_t r)
{
    const uint32_t u = __float_as_uint(x), mag = u & 0x7fffffffu;
    float a = __builtin_fabsf(x);
    if (!PLAIN)
        a = mag > kLimBits ? __uint_as_float(kLimBits) : a;
    const float q = a * inv;
    const uint32_t t = (q < 0x1p-6f ? __float_as_uint(q + 0x1p-6f) - (8u << 20) : __float_as_uint(q)) + (r << 4);
    uint32_t c = (t >> 20) - 960u;
    if (ROOT) {
        const uint32_t some = __float_as_uint(q) < 1u ? __float_as_uint(q) : 1u;
        c = c > some ? c : some;
    }
    if (!PLAIN)
        c = mag < kInf ? c : 0x7fu;
    return ROOT ? c : c | ((u >> 24) & 0x80u);
}

template <bool ROOT, bool PLAIN>
__device__ __forceinline__ uint2 code8(const float (&x)[8], const uint32_t (&r)[8], uint32_t byte)
{
    const float inv = inv_scale(byte);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 8; ++k)
        w[k >> 2] |= code_random<ROOT, PLAIN>(x[k], inv, ROOT ? r[k] >> 16 : r[k] & 0xffffu) << (8 * (k & 3));
    return make_uint2(w[0], w[1]);
}

// The codes of a lane's eight values and their block's exponent byte.
template <bool ROOT>
__device__ __forceinline__ uint2 encode(const float (&x)[8], const uint32_t (&r)[8], uint32_t &byte)
{
    uint32_t mx = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = ROOT ? __float_as_uint(x[k]) : __float_as_uint(x[k]) & 0x7fffffffu;
        mx = b > mx ? b : mx;
    }
    // all of a wave's values are numbers that bf16 holds, but for a step gone wrong
    if (__ballot(mx > kLimBits) == 0) {
        byte = block_byte(over_block(mx));
        return code8<ROOT, true>(x, r, byte);
    }
    mx = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const uint32_t b = mag_bits(x[k]);
        mx = b > mx ? b : mx;
    }
    byte = block_byte(over_block(mx));
    return code8<ROOT, false>(x, r, byte);
}

// The scalars of a step with 8-bit states.
struct SmallScalars {
    float b1, omb1, b2, omb2, eps, decay, wd;
    float rate;   // lr / bias1
    float per;    // 1 / sqrt(bias2)
    bool l2;
};

// adam1 with the quotient from the reciprocal and from the root that the state needs
// anyway: m_hat / (sqrt(v_hat) + eps) with v_hat = v / bias2 as m rate / (sqrt(v) per
// + eps).  m and v have adam1's bits; the quotient carries at most 8 roundings more
// (2^-21 of the update, which its codes' steps of 1/16 drown), and costs 40 issue slots
// less of 175 an element, where 126 keep up with memory.
__device__ __forceinline__ void adam_small(const SmallScalars &s, float g, float &p, float &m, float &v, float &root)
{
    p = p * s.decay;
    if (s.l2)
        g = g + s.wd * p;
    m = s.b1 * m + s.omb1 * g;
    v = s.b2 * v + s.omb2 * (g * g);
    root = sqrtf(v);
    const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(root, s.per, s.eps));
    p = __builtin_fmaf(-(m * s.rate), r, p);
}

template <bool SMALL>
__global__ __launch_bounds__(256) void tensors_kernel(const TensorArgs a)
{
    AdamScalars sc = a.sc;
    float rate = a.rate, per = a.per;
    int64_t step = a.step;
    if (a.table) {
        // a counter outside the table leaves every buffer as it is
        step = *a.counter;
        if (step < 1 || step > a.n_table)
            return;
        sc = a.table[step - 1];
        if (SMALL) {
            rate = sc.lr / sc.bias1;
            per = 1.0f / sqrtf(sc.bias2);
        }
    }
    const float coef = a.clip ? *a.clip : 1.0f;
    const int k0 = tensor_of(a, blockIdx.x);
    const Tensor &t = a.t[k0];
    sc.has_wd = sc.has_wd && (a.decay >> k0 & 1);
    const int64_t i = (int64_t)((int)blockIdx.x - a.tile0[k0]) * kTensorTile + threadIdx.x * 8;
    const int64_t left = t.n - i;
    const int n = left <= 0 ? 0 : left < 8 ? (int)left : 8;
    const bool vec = n == 8;
    float g[8], p[8], m[8], v[8];
    load8(t.grad, a.g_bf16, i, vec, n, g);
    load8(t.master, false, i, vec, n, p);
    if (SMALL) {
        // the codes of a lane are of one block
        uint32_t bm = 0, bv = 0;
        uint2 cm = make_uint2(0, 0), cv = cm;
        if (n > 0) {
            cm = load_bytes8(static_cast<const uint8_t *>(t.m) + i, vec, n);
            cv = load_bytes8(static_cast<const uint8_t *>(t.v) + i, vec, n);
            bm = t.ms[i >> 5];
            bv = t.vs[i >> 5];
        }
        bm *= 0x01010101u;
        bv *= 0x01010101u;
        decode8(cm, make_uint2(bm, bm), m);
        decode8(cv, make_uint2(bv, bv), v);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            v[k] = v[k] * v[k];
    } else {
        load8(t.m, false, i, vec, n, m);
        load8(t.v, false, i, vec, n, v);
    }
    if (SMALL) {
        SmallScalars ss;
        ss.b1 = sc.b1, ss.omb1 = sc.omb1, ss.b2 = sc.b2, ss.omb2 = sc.omb2, ss.eps = sc.eps, ss.wd = sc.wd;
        ss.decay = sc.has_wd && sc.decoupled ? sc.decay : 1.0f;
        ss.l2 = sc.has_wd && !sc.decoupled;
        ss.rate = rate, ss.per = per;
        const uint2 key = step_keys(a.seed, step);
        uint32_t r[8], bm, bv;
        float root[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            adam_small(ss, g[k] * coef, p[k], m[k], v[k], root[k]);
            r[k] = random_bits(key, t.number + i + k);
            if (k >= n)
                m[k] = root[k] = 0.0f;
        }
        const uint2 wm = encode<false>(m, r, bm), wv = encode<true>(root, r, bv);
        if (n == 0)
            return;
        store_bytes8(static_cast<uint8_t *>(t.m) + i, vec, n, wm);
        store_bytes8(static_cast<uint8_t *>(t.v) + i, vec, n, wv);
        if ((threadIdx.x & 3) == 0) {
            t.ms[i >> 5] = (uint8_t)bm;
            t.vs[i >> 5] = (uint8_t)bv;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            adam1(sc, g[k] * coef, p[k], m[k], v[k]);
        if (n == 0)
            return;
        store8(t.m, false, i, vec, n, m);
        store8(t.v, false, i, vec, n, v);
    }
    if (n == 0)
        return;
    store8(t.master, false, i, vec, n, p);
    if (t.param)
        store8(t.param, true, i, vec, n, p);
}

// The sum of squares of 8192 elements of a tensor's gradient, in fp64, where each
// square is exact.
__global__ __launch_bounds__(256) void tensors_sum_kernel(const TensorArgs a)
{
    __shared__ double part[4];
    const int k0 = tensor_of(a, blockIdx.x);
    const Tensor &t = a.t[k0];
    const int64_t i0 = (int64_t)((int)blockIdx.x - a.tile0[k0]) * kSumTile + threadIdx.x * 8;
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < kSumTile / 2048; ++j) {
        const int64_t i = i0 + 2048 * j, left = t.n - i;
        if (left <= 0)
            break;
        const int n = left < 8 ? (int)left : 8;
        float g[8];
        load8(t.grad, a.g_bf16, i, n == 8, n, g);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            s += (double)g[k] * (double)g[k];
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2)
        s += __shfl_xor(s, d, 64);
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = s;
    __syncthreads();
    if (threadIdx.x == 0)
        a.sums[a.first_sum + blockIdx.x] = ((part[0] + part[1]) + part[2]) + part[3];
}

// What 8-bit states stand for; `second`: the square, which is v.  Exact in bf16
// (a root has four bits, its square eight) down to fp32's smallest numbers.
__global__ __launch_bounds__(256) void state_read_kernel(int64_t n_all, const uint8_t *codes, const uint8_t *scales,
                                                         bool second, void *out, bool bf16)
{
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8, left = n_all - i;
    if (left <= 0)
        return;
    const int n = left < 8 ? (int)left : 8;
    const uint32_t b = scales[i >> 5] * 0x01010101u;
    float x[8];
    decode8(load_bytes8(codes + i, n == 8, n), make_uint2(b, b), x);
    if (second)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            x[k] *= x[k];
    store8(out, bf16, i, n == 8, n, x);
}

int64_t tensor_tiles(int64_t n, int tile) { return (n + tile - 1) / tile; }

zero_status check_tensors(int32_t n_tensors, const zero_tensor *ts, int32_t format, int32_t grad_dtype)
{
    if (n_tensors < 0 || (n_tensors > 0 && !ts))
        return fail(ZERO_ERR_INVALID_ARG, "a list of %d tensors is required", n_tensors);
    if (format != ZERO_STATE_FP32 && format != ZERO_STATE_E4M3)
        return fail(ZERO_ERR_INVALID_ARG, "unknown state format %d", format);
    if (!known_dtype(grad_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "unknown gradient dtype %d", grad_dtype);
    const bool small = format == ZERO_STATE_E4M3;
    for (int32_t k = 0; k < n_tensors; ++k) {
        const zero_tensor &t = ts[k];
        if (t.n < 0)
            return fail(ZERO_ERR_INVALID_ARG, "tensor %d: negative length", k);
        if (t.n > kMaxDim)
            return fail(ZERO_ERR_UNSUPPORTED, "tensor %d: too long", k);
        if (t.n == 0)
            continue;
        if (!t.master || !t.grad || !t.m || !t.v || (small && (!t.m_scales || !t.v_scales)))
            return fail(ZERO_ERR_INVALID_ARG, "tensor %d: master, grad, m, v%s are required", k,
                        small ? " and the scales" : "");
        if (!aligned(t.master, 4) || !aligned(t.grad, bytes_of(grad_dtype)) || !aligned(t.param, 2) ||
            (!small && (!aligned(t.m, 4) || !aligned(t.v, 4))))
            return fail(ZERO_ERR_ALIGNMENT, "tensor %d: a buffer is misaligned", k);
        const void *ms = small ? t.m_scales : nullptr, *vs = small ? t.v_scales : nullptr;
        if (is_one_of(t.master, {t.grad, t.param, t.m, t.v, ms, vs}) || is_one_of(t.grad, {t.param, t.m, t.v, ms, vs}) ||
            is_one_of(t.param, {t.m, t.v, ms, vs}) || is_one_of(t.m, {t.v, ms, vs}) || is_one_of(t.v, {ms, vs}) ||
            is_one_of(ms, {vs}))
            return fail(ZERO_ERR_INVALID_ARG, "tensor %d: its buffers need memory each", k);
    }
    return ZERO_OK;
}

// Launches `go(args, blocks)` for kTensors tensors at a time, the empty ones left
// out.
template <class F>
zero_status each_launch(int32_t n_tensors, const zero_tensor *ts, int32_t grad_dtype, int tile,
                        TensorArgs &a, const char *what, F go)
{
    constexpr int64_t kMost = int64_t(0xffffffffu) / 256;
    int64_t number = 0, tiles = 0, before = 0;
    a.g_bf16 = grad_dtype == ZERO_BF16;
    a.n_tensors = 0;
    a.decay = 0;
    (void)hipGetLastError();
    for (int32_t k = 0; k <= n_tensors; ++k) {
        const bool end = k == n_tensors;
        if (a.n_tensors > 0 && (end || a.n_tensors == kTensors || tiles + tensor_tiles(ts[k].n, tile) > kMost)) {
            a.first_sum = before;
            go(a, (unsigned)tiles);
            const zero_status st = launched(what);
            if (st != ZERO_OK)
                return st;
            before += tiles;
            tiles = 0;
            a.n_tensors = 0;
            a.decay = 0;
        }
        if (end)
            break;
        const zero_tensor &t = ts[k];
        if (t.n > 0) {
            a.tile0[a.n_tensors] = (int32_t)tiles;
            a.decay |= (uint64_t)(t.decay != 0) << a.n_tensors;
            Tensor &d = a.t[a.n_tensors++];
            d.master = t.master, d.grad = t.grad, d.param = t.param, d.m = t.m, d.v = t.v;
            d.ms = t.m_scales, d.vs = t.v_scales, d.n = t.n, d.number = number;
            tiles += tensor_tiles(t.n, tile);
        }
        number += (t.n + 31) / 32 * 32;
    }
    return ZERO_OK;
}

// No tensor may need more blocks than one launch has.
zero_status check_tiles(int32_t n_tensors, const zero_tensor *ts)
{
    for (int32_t k = 0; k < n_tensors; ++k)
        if (tensor_tiles(ts[k].n, kTensorTile) > int64_t(0xffffffffu) / 256)
            return fail(ZERO_ERR_UNSUPPORTED, "tensor %d: too long for one launch", k);
    return ZERO_OK;
}

zero_status run_tensors(int32_t n_tensors, const zero_tensor *ts, int32_t format, int32_t grad_dtype, TensorArgs &a,
                        hipStream_t s)
{
    const bool small = format == ZERO_STATE_E4M3;
    return each_launch(n_tensors, ts, grad_dtype, kTensorTile, a, "adam_tensors",
                       [&](const TensorArgs &args, unsigned blocks) {
                           if (small)
                               hipLaunchKernelGGL(tensors_kernel<true>, dim3(blocks), dim3(256), 0, s, args);
                           else
                               hipLaunchKernelGGL(tensors_kernel<false>, dim3(blocks), dim3(256), 0, s, args);
                       });
}

}  // namespace
}  // namespace zs

extern "C" {

zero_status zero_adam_tensors(int32_t n_tensors, const zero_tensor *tensors, int32_t state_format,
                              int32_t grad_dtype, const zero_adam_cfg *cfg, uint64_t seed,
                              const float *clip_coef, void *stream)
{
    using namespace zs;
    zero_status st;
    if (!cfg)
        return fail(ZERO_ERR_INVALID_ARG, "cfg is NULL");
    TensorArgs a;
    std::memset(&a, 0, offsetof(TensorArgs, t));
    zero_adam_table_entry e;
    if ((st = zero_adam_table_fill(cfg, 1, &e)) != ZERO_OK ||
        (st = check_tensors(n_tensors, tensors, state_format, grad_dtype)) != ZERO_OK ||
        (st = check_tiles(n_tensors, tensors)) != ZERO_OK)
        return st;
    if (!aligned(clip_coef, 4))
        return fail(ZERO_ERR_ALIGNMENT, "clip_coef is misaligned");
    std::memcpy(&a.sc, &e, sizeof e);
    a.rate = a.sc.lr / a.sc.bias1;
    a.per = 1.0f / std::sqrt(a.sc.bias2);
    a.step = cfg->step;
    a.seed = seed;
    a.clip = clip_coef;
    return run_tensors(n_tensors, tensors, state_format, grad_dtype, a, static_cast<hipStream_t>(stream));
}

zero_status zero_adam_tensors_table(int32_t n_tensors, const zero_tensor *tensors, int32_t state_format,
                                    int32_t grad_dtype, const zero_adam_table_entry *table, int64_t n_entries,
                                    const int64_t *step_counter, uint64_t seed, const float *clip_coef,
                                    void *stream)
{
    using namespace zs;
    zero_status st;
    if (!table || !step_counter || n_entries < 1)
        return fail(ZERO_ERR_INVALID_ARG, "table, step_counter and n_entries >= 1 are required");
    if (!aligned(table, 4) || !aligned(step_counter, 8) || !aligned(clip_coef, 4))
        return fail(ZERO_ERR_ALIGNMENT, "misaligned step table, counter or clip_coef");
    if ((st = check_tensors(n_tensors, tensors, state_format, grad_dtype)) != ZERO_OK ||
        (st = check_tiles(n_tensors, tensors)) != ZERO_OK)
        return st;
    TensorArgs a;
    std::memset(&a, 0, offsetof(TensorArgs, t));
    a.table = reinterpret_cast<const AdamScalars *>(table);
    a.counter = step_counter;
    a.n_table = n_entries;
    a.seed = seed;
    a.clip = clip_coef;
    return run_tensors(n_tensors, tensors, state_format, grad_dtype, a, static_cast<hipStream_t>(stream));
}

int64_t zero_tensors_partials_count(int32_t n_tensors, const zero_tensor *tensors)
{
    int64_t n = 0;
    for (int32_t k = 0; tensors && k < n_tensors; ++k)
        n += tensors[k].n > 0 ? zs::tensor_tiles(tensors[k].n, zs::kSumTile) : 0;
    return n;
}

zero_status zero_tensors_sumsq(int32_t n_tensors, const zero_tensor *tensors, int32_t grad_dtype, double *partials,
                               int64_t n_partials, void *stream)
{
    using namespace zs;
    zero_status st;
    if (n_tensors < 0 || (n_tensors > 0 && !tensors))
        return fail(ZERO_ERR_INVALID_ARG, "a list of %d tensors is required", n_tensors);
    if (!known_dtype(grad_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "unknown gradient dtype %d", grad_dtype);
    for (int32_t k = 0; k < n_tensors; ++k) {
        const zero_tensor &t = tensors[k];
        if (t.n < 0 || t.n > kMaxDim || (t.n > 0 && !t.grad))
            return fail(ZERO_ERR_INVALID_ARG, "tensor %d: a length in [0, 2^40] and a gradient are required", k);
        if (!aligned(t.grad, bytes_of(grad_dtype)))
            return fail(ZERO_ERR_ALIGNMENT, "tensor %d: the gradient is misaligned", k);
        if (t.grad && t.grad == partials)
            return fail(ZERO_ERR_INVALID_ARG, "tensor %d: the partial sums need memory of their own", k);
    }
    if ((st = check_tiles(n_tensors, tensors)) != ZERO_OK)
        return st;
    const int64_t need = zero_tensors_partials_count(n_tensors, tensors);
    if (need == 0)
        return ZERO_OK;
    if (!partials || n_partials < need)
        return fail(ZERO_ERR_INVALID_ARG, "%lld partial sums are required", (long long)need);
    if (!aligned(partials, 8))
        return fail(ZERO_ERR_ALIGNMENT, "partials is misaligned");
    TensorArgs a;
    std::memset(&a, 0, offsetof(TensorArgs, t));
    a.sums = partials;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return each_launch(n_tensors, tensors, grad_dtype, kSumTile, a, "tensors_sumsq",
                       [&](const TensorArgs &args, unsigned blocks) {
                           hipLaunchKernelGGL(tensors_sum_kernel, dim3(blocks), dim3(256), 0, s, args);
                       });
}

zero_status zero_adam_state_read(int64_t n, const uint8_t *codes, const uint8_t *scales, int32_t second, void *out,
                                 int32_t out_dtype, void *stream)
{
    using namespace zs;
    if (n < 0)
        return fail(ZERO_ERR_INVALID_ARG, "negative length");
    if (!known_dtype(out_dtype))
        return fail(ZERO_ERR_INVALID_ARG, "out: unknown dtype %d", out_dtype);
    if (n == 0)
        return ZERO_OK;
    if (!codes || !scales || !out)
        return fail(ZERO_ERR_INVALID_ARG, "codes, scales and out are required");
    if (!aligned(out, bytes_of(out_dtype)))
        return fail(ZERO_ERR_ALIGNMENT, "out is misaligned");
    if (is_one_of(out, {codes, scales}))
        return fail(ZERO_ERR_INVALID_ARG, "a state is not read back in place");
    const int64_t blocks = tensor_tiles(n, kTensorTile);
    if (blocks > int64_t(0xffffffffu) / 256)
        return fail(ZERO_ERR_UNSUPPORTED, "too long for one launch");
    (void)hipGetLastError();
    hipLaunchKernelGGL(state_read_kernel, dim3((unsigned)blocks), dim3(256), 0, static_cast<hipStream_t>(stream), n,
                       codes, scales, second != 0, out, out_dtype == ZERO_BF16);
    return launched("adam_state_read");
}

}  // extern "C"
