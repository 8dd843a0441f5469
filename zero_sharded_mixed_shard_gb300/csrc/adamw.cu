// AdamW over many separate tensors (moments in 32 or in 8 bits) and the
// global gradient norm, each in one launch over a planned list of tensors.
//
// The plan cuts every tensor into chunks; a table in device memory holds one
// record per tensor and the running count of chunks, so a CTA finds the
// tensor of chunk c by bisection and a launch needs no per-tensor host work.
// Both operators stream each byte once and are bound by HBM: with 16-bit
// gradients and parameters a step moves 2P + 26 bytes per element with fp32
// moments and 2P + 14 + 1/16 with 8-bit ones, the norm 2P.
//
// Mathematics: AdamW (I. Loshchilov, F. Hutter, Decoupled Weight Decay
// Regularization) with the bias corrections folded into two factors; 8-bit
// moments by blocks of 256 that share a scale (block-wise quantisation,
// T. Dettmers et al.), the momentum to the nearest code, the root of the
// variance at random between its two neighbours.  The variance moves by a
// thousandth a step, far less than a code's step (up to an eighth), so rounded
// to the nearest it would stand still.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "zero_train.h"

// Defined in step.cu (not exported): keeps zero_last_cuda_error current.
__attribute__((visibility("hidden"))) int zero_record_cuda_error(int err);

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;                    // elements of a warp's unit, and of an 8-bit scale
constexpr int kChunk = kWarps * kBlock;        // elements of a CTA's unit of the step
constexpr int kNormVecs = 4;                   // 8-element vectors of a thread in a chunk of the norm; 1 in a short list
constexpr int kNormStep = kThreads * 8;        // elements of a chunk for each of them
constexpr int kShortNorm = 400;                // chunks (of 4) up to which a list counts as short
constexpr int kMaxPartials = 2048;             // CTAs of the norm at most
constexpr float kMax8 = 448.0f;                // largest E4M3 value
constexpr float kInvMax8 = 1.0f / 448.0f;
constexpr float kTiny = 1.262177448353619e-29f; // 2^-96
constexpr float kLowSquares = 8.271806125530277e-25f;  // 2^-80
constexpr float kHighSquares = 1.2676506002282294e30f; // 2^100

struct Tensor {
    const void* g;
    long long stride;
    float* w;
    void* m;
    void* v;
    float* ms;
    float* vs;
    void* p;
    long long n;
    float decay;     // weight_decay
    float lr_scale;
    int phase;       // elements between the preceding vector boundary and element 0, or -1: streams differ
    int gphase;      // the same for the gradients alone
};

// The device table: this header, the running chunk counts of the step and of
// the norm (n_tensors + 1 each), then the tensors' records.
struct Header {
    unsigned int ticket; // CTAs of the running norm that are done; 0 between calls
    unsigned int pad[3];
    double partial[kMaxPartials];
};

struct Args {
    Header* head;
    const long long* first;  // [n_tensors + 1] first chunk of each tensor
    const Tensor* tensors;
    int n_tensors;
    int P;
    int p_pow2;
    float inv_p;
    long long chunks;
    const float* stats;
    float lr, b1, b2, omb1, omb2, r1, c2, eps;
    unsigned int seed;
    int stages, stage_bytes; // pipeline kernel
    float grad_scale, max_norm;
    float* out;
};

// ---------------------------------------------------------------------------
// Device helpers
// ---------------------------------------------------------------------------

// MurmurHash3's 32-bit finaliser (A. Appleby): every input bit reaches every
// output bit, which is all that rounding needs.
__host__ __device__ __forceinline__ unsigned int mix32(unsigned int h)
{
    h = (h ^ (h >> 16)) * 0x85ebca6bu;
    h = (h ^ (h >> 13)) * 0xc2b2ae35u;
    return h ^ (h >> 16);
}

template <int T> struct Elem;
template <> struct Elem<ZERO_TYPE_FP16> { using type = __half; };
template <> struct Elem<ZERO_TYPE_BF16> { using type = __nv_bfloat16; };
template <> struct Elem<ZERO_TYPE_FP32> { using type = float; };

__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

template <int T> __device__ __forceinline__ unsigned int pack2(float a, float b)
{
    if constexpr (T == ZERO_TYPE_FP16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const unsigned int*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const unsigned int*>(&h);
    }
}

template <int T> __device__ __forceinline__ float2 unpack2(unsigned int u)
{
    if constexpr (T == ZERO_TYPE_FP16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
    else return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// Eight consecutive gradients as loaded: one 16-byte access, two for fp32.
template <int T> struct Raw8 {
    uint4 a[T == ZERO_TYPE_FP32 ? 2 : 1];
};

template <int T> __device__ __forceinline__ Raw8<T> load8(const void* p)
{
    Raw8<T> r;
    const uint4* q = static_cast<const uint4*>(p);
    r.a[0] = __ldcs(q);
    if constexpr (T == ZERO_TYPE_FP32) r.a[1] = __ldcs(q + 1);
    return r;
}

template <int T> __device__ __forceinline__ void set8(float (&v)[8], const Raw8<T>& r)
{
    const unsigned int u[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (T == ZERO_TYPE_FP32) {
            const unsigned int w[4] = {r.a[1].x, r.a[1].y, r.a[1].z, r.a[1].w};
            v[j] = __uint_as_float(u[j]);
            v[4 + j] = __uint_as_float(w[j]);
        } else {
            const float2 f = unpack2<T>(u[j]);
            v[2 * j] = f.x;
            v[2 * j + 1] = f.y;
        }
    }
}

template <int T> __device__ __forceinline__ void add8(float (&acc)[8], const Raw8<T>& r)
{
    const unsigned int u[4] = {r.a[0].x, r.a[0].y, r.a[0].z, r.a[0].w};
    if constexpr (T == ZERO_TYPE_FP32) {
        const unsigned int w[4] = {r.a[1].x, r.a[1].y, r.a[1].z, r.a[1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            acc[j] = __fadd_rn(acc[j], __uint_as_float(u[j]));
            acc[4 + j] = __fadd_rn(acc[4 + j], __uint_as_float(w[j]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = unpack2<T>(u[j]);
            acc[2 * j] = __fadd_rn(acc[2 * j], f.x);
            acc[2 * j + 1] = __fadd_rn(acc[2 * j + 1], f.y);
        }
    }
}

// x / d from r close to 1 / d: the quotient x r and one correction step by its
// exact remainder (P. Markstein, IBM J. Res. Dev. 34(1), 1990).  For x a sum of
// gradients and d a number of ranks the result is the correctly rounded one
// (zero_selftest_mean_division) unless it is below fp32's normal range.  It
// has no rare path, unlike CUDA's division, whose call costs the step's loop
// its registers.
__device__ __forceinline__ float divide(float x, float d, float r)
{
    const float q = __fmul_rn(x, r);
    const float c = __fmaf_rn(__fmaf_rn(-q, d, x), r, q);
    return fabsf(q) < __int_as_float(0x7f800000) ? c : q; // an infinite quotient has no remainder
}

__device__ __forceinline__ float mean_of(float sum, const Args& a)
{
    if (a.P == 1) return sum;
    return a.p_pow2 ? __fmul_rn(sum, a.inv_p) : divide(sum, static_cast<float>(a.P), a.inv_p);
}

// The tensor that chunk c belongs to: the last one whose first chunk is <= c
// (tensors without elements have no chunk and are never the last such one).
// A warp looks at 32 places at once: two dependent reads find one of a
// thousand tensors.
__device__ __forceinline__ int find_tensor(const long long* first, int n, long long c)
{
    const int lane = threadIdx.x & 31;
    int lo = 0;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const unsigned int before = __ballot_sync(0xffffffffu, at < n && __ldg(first + lo + at) <= c);
        const int skip = (__popc(before) - 1) * step; // lane 0's place is always before
        lo += skip;
        n = min(step, n - skip);
    }
    return lo;
}

// Programmatic launch: the wait returns when the preceding kernel is complete
// and its writes are visible; nothing is read before it.
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float fast_sqrt(float x)
{
    float y;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x)); // relative error at most 2^-23
    return y;
}

// The root correctly rounded from the approximate one, s = x y: s plus half of
// y times the exact remainder x - s^2 (P. Markstein, as above).  A stored code
// follows from the root's bits, so that a step on equal states gives equal
// codes wherever the same fp32 operations are done.  x is 0 or at least 2^-101,
// where the remainder, a multiple of x 2^-48 or more, is still exact, and finite.
__device__ __forceinline__ float exact_sqrt(float x)
{
    float y;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(x, 1.17549435e-38f)));
    const float s = __fmul_rn(x, y);
    return __fmaf_rn(__fmaf_rn(-s, s, x), __fmul_rn(0.5f, y), s);
}

// The same for any x >= 0: what is below 2^-96 is scaled by 2^64, its root by
// 2^-32 (both exact; the smallest root is above 2^-75), and infinity, whose
// remainder is no number, is its own root.
__device__ __forceinline__ float exact_sqrt_any(float x)
{
    const bool low = x < kTiny;
    const float s = exact_sqrt(low ? __fmul_rn(x, 1.8446744073709552e19f) : x);
    if (x == __int_as_float(0x7f800000)) return x;
    return low ? __fmul_rn(s, 2.3283064365386963e-10f) : s;
}

__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x)); // 1 ulp
    return y;
}

__device__ __forceinline__ float max_or_nan(float x, float y)
{
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__device__ __forceinline__ float min_or_nan(float x, float y)
{
    float z;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

// 448 / a correctly rounded: the reciprocal refined to the nearest one, then
// the quotient.  Above 2^120 both sides are scaled by 2^-8 (exact): the
// reciprocal of what is above 2^126 would be flushed to 0.
__device__ __forceinline__ float scale_inverse(float a)
{
    const float f = a > 1.329227995784916e36f ? 0.00390625f : 1.0f;
    a *= f;
    const float r = fast_rcp(a);
    return divide(kMax8 * f, a, __fmaf_rn(__fmaf_rn(-a, r, 1.0f), r, r));
}

// ---------------------------------------------------------------------------
// The step
// ---------------------------------------------------------------------------

// What a warp knows of its block of 256 elements besides the elements.
struct Block {
    float lr, decay, factor;
    unsigned int key;    // of the tensor and the seed
    float ms, vs;        // 8-bit moments: the block's scales, and where the new ones go
    float* ms_out;
    float* vs_out;
};

// The update of a lane's eight elements in registers.  g: sums over the
// ranks.  With 8-bit moments mc, vc hold the codes and receive the new ones;
// the whole warp calls it, and `pair(j)` is element j's place in its tensor's
// pairs, `odd(j)` its place in the pair.
template <int BITS, bool ONE, class Pair, class Odd>
__device__ __forceinline__ void update(const Args& a, const Block& k, float (&w)[8], float (&m)[8],
                                       float (&v)[8], const float (&g)[8], unsigned int (&mc)[2], unsigned int (&vc)[2],
                                       Pair pair, Odd odd)
{
    if constexpr (BITS == 8) {
        const float ms = k.ms, vs = k.vs;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const unsigned short cm = static_cast<unsigned short>(mc[q >> 1] >> (16 * (q & 1)));
            const unsigned short cv = static_cast<unsigned short>(vc[q >> 1] >> (16 * (q & 1)));
            const float2 fm = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(cm, __NV_E4M3)));
            const float2 fv = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(cv, __NV_E4M3)));
            m[2 * q] = __fmul_rn(fm.x, ms);
            m[2 * q + 1] = __fmul_rn(fm.y, ms);
            const float rx = __fmul_rn(fv.x, vs), ry = __fmul_rn(fv.y, vs);
            v[2 * q] = __fmul_rn(rx, rx);
            v[2 * q + 1] = __fmul_rn(ry, ry);
        }
    }
    float high_m = 0.0f, high_r = 0.0f; // largest magnitudes, or NaN
    float low_v = kTiny, high_v = 0.0f;
    const float minus_rate = -__fmul_rn(k.lr, a.r1);
    auto weight = [&](int j, float root) {
        const float inv = fast_rcp(__fmaf_rn(root, a.c2, a.eps));
        w[j] = __fmaf_rn(-k.decay, w[j], w[j]);
        w[j] = __fmaf_rn(__fmul_rn(m[j], minus_rate), inv, w[j]);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float gg = __fmul_rn(ONE ? g[j] : mean_of(g[j], a), k.factor);
        m[j] = __fadd_rn(__fmul_rn(m[j], a.b1), __fmul_rn(gg, a.omb1));
        v[j] = __fadd_rn(__fmul_rn(v[j], a.b2), __fmul_rn(__fmul_rn(gg, gg), a.omb2));
        if constexpr (BITS == 8) {
            low_v = fminf(low_v, v[j]);
            high_v = fmaxf(high_v, v[j]);
        } else {
            weight(j, fast_sqrt(v[j]));
        }
    }
    if constexpr (BITS == 8) { // the rare values (zeros among them) apart: one branch for a lane's eight
        if (low_v < kTiny || high_v == __int_as_float(0x7f800000)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = exact_sqrt_any(v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = exact_sqrt(v[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            weight(j, v[j]);
            high_m = max_or_nan(high_m, fabsf(m[j]));
            high_r = max_or_nan(high_r, v[j]);
        }
    }
    if constexpr (BITS == 8) {
        // as bits the magnitudes are ordered like the values, NaN above infinity
        const float am = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(high_m) & 0x7fffffffu));
        const float ar = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(high_r) & 0x7fffffffu));
        const float im = am < kTiny ? 0.0f : scale_inverse(am), ir = ar < kTiny ? 0.0f : scale_inverse(ar);
        if ((threadIdx.x & 31) == 0) {
            const float nan = __int_as_float(0x7fffffff);
            *k.ms_out = am < kTiny ? 0.0f : isfinite(am) ? __fmul_rn(am, kInvMax8) : nan;
            *k.vs_out = ar < kTiny ? 0.0f : isfinite(ar) ? __fmul_rn(ar, kInvMax8) : nan;
        }
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const unsigned int lo = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(m[4 * q], im), __fmul_rn(m[4 * q + 1], im)),
                                                             __NV_SATFINITE, __NV_E4M3);
            const unsigned int hi = __nv_cvt_float2_to_fp8x2(make_float2(__fmul_rn(m[4 * q + 2], im), __fmul_rn(m[4 * q + 3], im)),
                                                             __NV_SATFINITE, __NV_E4M3);
            mc[q] = lo + (hi << 16);
        }
        unsigned int h = 0, code[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            // Sixteen random bits for each element, one hash for a pair.
            if (j == 0 || pair(j) != pair(j - 1)) h = mix32(pair(j) + k.key);
            const unsigned int random = odd(j) ? h >> 16 : h & 0xffffu;
            // Scaled by 2^-120 a value's E4M3 code is the top of its binary32
            // form (bits 30..20; E4M3's subnormals are fp32's), and adding
            // random bits below bit 20 before cutting there rounds up with
            // the probability of what is cut.  A zero stays 0, a root above
            // zero is at least 1, and the largest, 448, has no bits below its
            // code 0x7e (a block with the scale NaN may hold any codes).
            const float y = __fmul_rn(v[j], ir);
            const unsigned int cut = (__float_as_uint(__fmul_rn(y, 7.52316384526264e-37f)) + (random << 4)) >> 20;
            code[j] = max(cut, min(__float_as_uint(y), 1u));
        }
#pragma unroll
        for (int q = 0; q < 2; ++q)
            vc[q] = (code[4 * q] + (code[4 * q + 1] << 8)) + ((code[4 * q + 2] << 16) + (code[4 * q + 3] << 24));
    }
}

// A block at a tensor's end, or of a tensor whose streams do not share one
// phase: lane l has elements l, l + 32, ..., one access each.  Kept out of the
// main path's registers.
template <int GT, int PT, int BITS>
__device__ __noinline__ void step_by_elements(const Args& a, const Tensor* x, float lr, float decay, float factor,
                                               unsigned int key, long long b0, float go)
{
    using G = typename Elem<GT>::type;
    const long long n = x->n, stride = x->stride, first = b0 + (threadIdx.x & 31);
    Block k{lr, decay, factor, key, 0.0f, 0.0f, nullptr, nullptr};
    if constexpr (BITS == 8) {
        k.ms_out = x->ms + b0 / kBlock;
        k.vs_out = x->vs + b0 / kBlock;
        k.ms = *k.ms_out;
        k.vs = *k.vs_out;
    }
    float w[8], m[8], v[8], g[8];
    unsigned int mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long i = first + j * 32;
        w[j] = m[j] = v[j] = g[j] = 0.0f;
        if (i < 0 || i >= n) continue;
        w[j] = x->w[i];
        if constexpr (BITS == 32) {
            m[j] = static_cast<const float*>(x->m)[i];
            v[j] = static_cast<const float*>(x->v)[i];
        } else {
            mc[j >> 2] |= static_cast<unsigned int>(static_cast<const unsigned char*>(x->m)[i]) << (8 * (j & 3));
            vc[j >> 2] |= static_cast<unsigned int>(static_cast<const unsigned char*>(x->v)[i]) << (8 * (j & 3));
        }
        g[j] = to_float(static_cast<const G*>(x->g)[i]);
    }
    for (int r = 1; r < a.P; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const long long i = first + j * 32;
            if (i >= 0 && i < n) g[j] = __fadd_rn(g[j], to_float(static_cast<const G*>(x->g)[r * stride + i]));
        }
    if (go == 0.0f) return;
    update<BITS, false>(a, k, w, m, v, g, mc, vc, [&](int j) { return static_cast<unsigned int>((first + j * 32) >> 1); },
                        [&](int) { return (first & 1) != 0; });
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const long long i = first + j * 32;
        if (i < 0 || i >= n) continue;
        x->w[i] = w[j];
        if constexpr (BITS == 32) {
            static_cast<float*>(x->m)[i] = m[j];
            static_cast<float*>(x->v)[i] = v[j];
        } else {
            static_cast<unsigned char*>(x->m)[i] = static_cast<unsigned char>(mc[j >> 2] >> (8 * (j & 3)));
            static_cast<unsigned char*>(x->v)[i] = static_cast<unsigned char>(vc[j >> 2] >> (8 * (j & 3)));
        }
        static_cast<unsigned short*>(x->p)[i] = static_cast<unsigned short>(pack2<PT>(w[j], 0.0f));
    }
}

// One warp per block of 256 elements.  Where a tensor's streams share one
// 16-byte phase a lane owns 8 consecutive elements (whole-vector accesses);
// the blocks at its ends, and every block of other tensors, go element by
// element.  The two differ in which lane holds an element and in nothing
// else: results are the same.
// Bound by HBM on large lists, by the launch and three dependent reads (place,
// tensor, elements) on small ones.  Three CTAs an SM: at four the main path's
// registers spill (P = 2, 2.0e8 elements 1019 against 900 us).  At three the
// instances with 16-bit gradients keep theirs (fp16, 8-bit moments and several
// ranks: 4 bytes); fp32 gradients of several ranks spill 88 bytes with 32-bit
// moments and 64 with 8-bit ones.  Measured: eight bf16
// ranks of 2.0e8 parameters 1.30 ms (6500 GB/s, 0.958 of the measured copy
// bandwidth), 50 thousand parameters 6.2 us, 4.0e6 parameters of odd sizes with
// 8-bit moments and fp32 gradients 18.2 us (3940 GB/s; 16 us where one list's 72
// MB stay in L2).
template <int GT, int PT, int BITS, bool ONE>
__global__ void __launch_bounds__(kThreads, 3) zero_adamw_kernel(const __grid_constant__ Args a)
{
    using G = typename Elem<GT>::type;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    let_successor_start();
    wait_for_predecessor();
    Block k;
    float go = 1.0f;
    k.factor = 1.0f;
    if (a.stats) {
        k.factor = a.stats[1];
        go = a.stats[2];
    }
    // The place of the CTA's next chunk, looked up while the current one's loads are in flight.
    long long c = blockIdx.x, lo = 0, hi = 0, n = 0;
    int phase = 0;
    const Tensor* x = nullptr;
    auto look_up = [&] {
        if (c >= a.chunks || c < hi) return;
        const int ti = find_tensor(a.first, a.n_tensors, c);
        lo = __ldg(a.first + ti);
        hi = __ldg(a.first + ti + 1);
        x = a.tensors + ti;
        n = x->n;
        phase = x->phase;
        k.lr = __fmul_rn(a.lr, x->lr_scale);
        k.decay = __fmul_rn(k.lr, x->decay);
        k.key = BITS == 8 ? mix32(mix32(a.seed) + 0x9e3779b9u * static_cast<unsigned int>(ti + 1)) : 0u;
    };
    look_up();
    while (c < a.chunks) {
        const long long b0 = (c - lo) * kChunk + warp * kBlock - max(phase, 0); // the block's first element
        c += gridDim.x;
        if (b0 >= n) {
            look_up();
            continue;
        }
        if (phase < 0 || b0 < 0 || b0 + kBlock > n) {
            step_by_elements<GT, PT, BITS>(a, x, k.lr, k.decay, k.factor, k.key, b0, go);
            if (go == 0.0f) return;
            look_up();
            continue;
        }
        const long long i0 = b0 + lane * 8;
        float w[8], m[8], v[8], g[8];
        unsigned int mc[2] = {0u, 0u}, vc[2] = {0u, 0u}; // 8-bit codes
        float4* wp = reinterpret_cast<float4*>(x->w + i0);
        *reinterpret_cast<float4*>(w) = __ldcs(wp);
        *reinterpret_cast<float4*>(w + 4) = __ldcs(wp + 1);
        if constexpr (BITS == 32) {
            const float4* mp = reinterpret_cast<const float4*>(static_cast<float*>(x->m) + i0);
            const float4* vp = reinterpret_cast<const float4*>(static_cast<float*>(x->v) + i0);
            *reinterpret_cast<float4*>(m) = __ldcs(mp);
            *reinterpret_cast<float4*>(m + 4) = __ldcs(mp + 1);
            *reinterpret_cast<float4*>(v) = __ldcs(vp);
            *reinterpret_cast<float4*>(v + 4) = __ldcs(vp + 1);
        } else {
            const uint2 mm = __ldcs(reinterpret_cast<const uint2*>(static_cast<unsigned char*>(x->m) + i0));
            const uint2 vv = __ldcs(reinterpret_cast<const uint2*>(static_cast<unsigned char*>(x->v) + i0));
            mc[0] = mm.x, mc[1] = mm.y, vc[0] = vv.x, vc[1] = vv.y;
            k.ms_out = x->ms + b0 / kBlock; // blocks start on multiples of 256 here
            k.vs_out = x->vs + b0 / kBlock;
            k.ms = *k.ms_out;
            k.vs = *k.vs_out;
        }
        const G* gp = static_cast<const G*>(x->g) + i0;
        if constexpr (ONE) {
            set8<GT>(g, load8<GT>(gp));
        } else {
            const long long stride = x->stride;
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = 0.0f;
            int r = 0;
            for (; r + 4 <= a.P; r += 4) {
                Raw8<GT> raw[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) raw[q] = load8<GT>(gp + (r + q) * stride);
#pragma unroll
                for (int q = 0; q < 4; ++q) add8<GT>(g, raw[q]);
            }
            for (; r < a.P; ++r) add8<GT>(g, load8<GT>(gp + r * stride));
        }
        if (go == 0.0f) return; // a gradient overflowed: nothing is written
        const Block now = k;
        float* mp_out = static_cast<float*>(x->m);
        float* vp_out = static_cast<float*>(x->v);
        unsigned short* p_out = static_cast<unsigned short*>(x->p) + i0;
        look_up();
        update<BITS, ONE>(a, now, w, m, v, g, mc, vc, [&](int j) { return static_cast<unsigned int>(i0 >> 1) + (j >> 1); },
                          [](int j) { return (j & 1) != 0; });
        __stcs(wp, *reinterpret_cast<float4*>(w));
        __stcs(wp + 1, *reinterpret_cast<float4*>(w + 4));
        if constexpr (BITS == 32) {
            float4* mp = reinterpret_cast<float4*>(mp_out + i0);
            float4* vp = reinterpret_cast<float4*>(vp_out + i0);
            __stcs(mp, *reinterpret_cast<float4*>(m));
            __stcs(mp + 1, *reinterpret_cast<float4*>(m + 4));
            __stcs(vp, *reinterpret_cast<float4*>(v));
            __stcs(vp + 1, *reinterpret_cast<float4*>(v + 4));
        } else {
            __stcs(reinterpret_cast<uint2*>(reinterpret_cast<unsigned char*>(mp_out) + i0), make_uint2(mc[0], mc[1]));
            __stcs(reinterpret_cast<uint2*>(reinterpret_cast<unsigned char*>(vp_out) + i0), make_uint2(vc[0], vc[1]));
        }
        __stcs(reinterpret_cast<uint4*>(p_out),
               make_uint4(pack2<PT>(w[0], w[1]), pack2<PT>(w[2], w[3]), pack2<PT>(w[4], w[5]), pack2<PT>(w[6], w[7])));
    }
}

// ---------------------------------------------------------------------------
// The step as a pipeline of bulk copies
// ---------------------------------------------------------------------------

// One CTA per SM.  A warp copies whole chunks (2048 elements of master, m, v
// and every rank's gradients) into a ring of shared-memory stages; groups of
// eight warps take the chunks in turn, a warp a block of 256, hand the stage
// back as soon as they have read it, and store their results directly.  The
// copies in flight do not depend on the warps' registers or on how far their
// arithmetic has come, which is what bounds the vector kernel.
// Measured, 1.3e9 parameters, P = 1: 32-bit moments 5.50 ms (6620 GB/s, 0.975 of
// the measured copy bandwidth; vector kernel 6.2 ms), 8-bit ones 3.29 ms (6350
// GB/s, 0.936; vector kernel 3.7 ms), where the arithmetic, about 75
// instructions an element, takes nearly the time of the bytes.
constexpr int kGroups = 3;
constexpr int kPipeThreads = 32 + kGroups * kThreads;
// A multiple of the groups: a stage always goes to the same group, which so
// waits for each of its fills in turn (a wait tells a fill from the next one
// only by parity).
constexpr int kMaxStages = 15;
constexpr int kPipeSmem = 224 * 1024;
// More copies in flight than this cost the stores (32-bit moments, P = 1: 3
// stages of 28 KB 6620 GB/s, 6 stages 6410), fewer leave reads waiting (8-bit,
// fp32 gradients: 3 stages of 20 KB 5510 GB/s, 6 stages 6730).
constexpr int kPipeTarget = 112 * 1024;
static_assert(kMaxStages % kGroups == 0, "stages by groups");
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_adamw_timeouts;

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ bool mbar_try(uint64_t* bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(smem_addr(bar)), "r"(parity)
                 : "memory");
    return done != 0;
}

// Waits for the phase of the given parity; false when two seconds have passed
// or another warp has given up.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int round = 0; round < (1 << 22); ++round) {
        for (int k = 0; k < 64; ++k)
            if (mbar_try(bar, parity)) return true;
        if (abort && *abort) return false;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 > kWaitLimitNs) break;
    }
    if (abort && atomicExch(const_cast<int*>(abort), 1) == 0) atomicAdd(&g_adamw_timeouts, 1u);
    return false;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    return mbar_try(bar, parity) || wait_slow(bar, parity, abort);
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(src), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "elect.sync _|q, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// What the copying warp says about a stage's chunk.
struct Chunk {
    const Tensor* x;
    float* w;
    void* m;
    void* v;
    void* p;
    float* ms;
    float* vs;
    long long n;
    long long b0;        // first element of its first block (may be negative)
    int from, to;        // blocks that are in the stage; the others go element by element
    float lr, decay;
    unsigned int key;
};

// STARVED: the instance of zero_selftest_adamw_wait alone.  Its first CTA never
// hands a stage back, and half of the copying warp's lanes ask for a phase that
// is over, so that the lanes of one warp get different answers.
template <int GT, int PT, int BITS, bool ONE, bool STARVED = false>
__global__ void __launch_bounds__(kPipeThreads, 1) zero_adamw_pipeline_kernel(const __grid_constant__ Args a)
{
    using G = typename Elem<GT>::type;
    constexpr int kGrad = kChunk * static_cast<int>(sizeof(G)); // bytes of a rank's row, of a moment's
    constexpr int kMoment = kChunk * BITS / 8;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ Chunk meta[kMaxStages];
    __shared__ int abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    volatile int* abort = &abort_flag;
    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&full[s])), "r"(1) : "memory");
            asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(&empty[s])), "r"(kWarps) : "memory");
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async;" ::: "memory");
    }
    __syncthreads();
    let_successor_start();
    wait_for_predecessor();
    float factor = 1.0f;
    if (a.stats) {
        factor = a.stats[1];
        if (a.stats[2] == 0.0f) return; // a gradient overflowed: nothing is written
    }
    if (warp == 0) {
        long long lo = 0, hi = 0, n = 0, stride = 0;
        Tensor x{};
        Chunk k{};
        int it = 0;
        bool ok = true;
        for (long long c = blockIdx.x; ok && c < a.chunks; c += gridDim.x, ++it) {
            if (c >= hi) {
                const int ti = find_tensor(a.first, a.n_tensors, c);
                lo = __ldg(a.first + ti);
                hi = __ldg(a.first + ti + 1);
                k.x = a.tensors + ti;
                x = *k.x;
                n = x.n;
                stride = x.stride;
                k.w = x.w, k.m = x.m, k.v = x.v, k.p = x.p, k.ms = x.ms, k.vs = x.vs, k.n = n;
                k.lr = __fmul_rn(a.lr, x.lr_scale);
                k.decay = __fmul_rn(k.lr, x.decay);
                k.key = BITS == 8 ? mix32(mix32(a.seed) + 0x9e3779b9u * static_cast<unsigned int>(ti + 1)) : 0u;
            }
            const int s = it % a.stages;
            uint32_t parity = ((it / a.stages) & 1) ^ 1;
            if (STARVED && blockIdx.x == 0 && it >= a.stages && lane >= 16) parity ^= 1;
            // one answer for the warp: below it works together, and so it must give up together
            ok = __all_sync(0xffffffffu, wait(&empty[s], parity, abort));
            if (!ok) break;
            k.b0 = (c - lo) * kChunk - max(x.phase, 0);
            k.from = k.b0 < 0 ? 1 : 0;
            k.to = static_cast<int>(max(0ll, min(static_cast<long long>(kWarps), (n - k.b0) / kBlock)));
            if (x.phase < 0 || k.to <= k.from) k.from = k.to = 0;
            const long long e0 = k.b0 + k.from * kBlock;
            const uint32_t count = static_cast<uint32_t>(k.to - k.from) * kBlock;
            if (lane == 0) {
                meta[s] = k;
                const uint32_t bytes = count * (4 + BITS / 4 + static_cast<uint32_t>(sizeof(G)) * a.P);
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(&full[s])), "r"(bytes)
                             : "memory");
            }
            __syncwarp();
            // One elected lane issues the rows: the copy instruction takes uniform registers, and under a condition on the
            // lane each would cost several hundred cycles.
            if (count > 0 && elect_one()) {
                unsigned char* st = smem + s * a.stage_bytes;
                const int at = k.from * kBlock;
                bulk_load(st + at * 4, x.w + e0, count * 4, &full[s]);
                st += kChunk * 4;
                bulk_load(st + at * BITS / 8, static_cast<unsigned char*>(x.m) + e0 * (BITS / 8), count * (BITS / 8), &full[s]);
                st += kMoment;
                bulk_load(st + at * BITS / 8, static_cast<unsigned char*>(x.v) + e0 * (BITS / 8), count * (BITS / 8), &full[s]);
                st += kMoment + at * sizeof(G);
                const G* g = static_cast<const G*>(x.g) + e0;
                for (int r = 0; r < (ONE ? 1 : a.P); ++r, st += kGrad, g += stride)
                    bulk_load(st, g, count * static_cast<uint32_t>(sizeof(G)), &full[s]);
            }
            __syncwarp();
        }
        if (!ok) // the copies in flight land before the CTA ends
            for (int k2 = max(0, it - a.stages); k2 < it; ++k2) wait_slow(&full[k2 % a.stages], (k2 / a.stages) & 1, nullptr);
        return;
    }
    const int group = (warp - 1) / kWarps, mine = (warp - 1) % kWarps;
    auto hand_back = [&](int s) {
        __syncwarp();
        if (lane == 0 && !(STARVED && blockIdx.x == 0))
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(&empty[s])) : "memory");
    };
    int it = 0;
    for (long long c = blockIdx.x; c < a.chunks; c += gridDim.x, ++it) {
        if (it % kGroups != group) continue;
        const int s = it % a.stages;
        const bool ok = wait(&full[s], (it / a.stages) & 1, abort);
        if (!__all_sync(0xffffffffu, ok)) break;
        const Chunk ch = meta[s];
        const long long b0 = ch.b0 + mine * kBlock;
        if (mine < ch.from || mine >= ch.to) {
            hand_back(s);
            if (b0 < ch.n) step_by_elements<GT, PT, BITS>(a, ch.x, ch.lr, ch.decay, factor, ch.key, b0, 1.0f);
            continue;
        }
        Block k{ch.lr, ch.decay, factor, ch.key, 0.0f, 0.0f, nullptr, nullptr};
        if constexpr (BITS == 8) {
            k.ms_out = ch.ms + b0 / kBlock;
            k.vs_out = ch.vs + b0 / kBlock;
            k.ms = *k.ms_out;
            k.vs = *k.vs_out;
        }
        // lane l has elements 4 l .. 4 l + 3 of each half of the block: accesses of 16 bytes (fp32) side by side
        const unsigned char* st = smem + s * a.stage_bytes;
        const int at = mine * kBlock + lane * 4;
        float w[8], m[8], v[8], g[8];
        unsigned int mc[2] = {0u, 0u}, vc[2] = {0u, 0u};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int e = at + h * 128;
            *reinterpret_cast<float4*>(w + 4 * h) = *reinterpret_cast<const float4*>(st + e * 4);
            if constexpr (BITS == 32) {
                *reinterpret_cast<float4*>(m + 4 * h) = *reinterpret_cast<const float4*>(st + (kChunk + e) * 4);
                *reinterpret_cast<float4*>(v + 4 * h) = *reinterpret_cast<const float4*>(st + (2 * kChunk + e) * 4);
            } else {
                mc[h] = *reinterpret_cast<const unsigned int*>(st + kChunk * 4 + e);
                vc[h] = *reinterpret_cast<const unsigned int*>(st + kChunk * 4 + kMoment + e);
            }
        }
        const unsigned char* gr = st + kChunk * 4 + 2 * kMoment + at * sizeof(G);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 0.0f;
#pragma unroll 4
        for (int r = 0; r < (ONE ? 1 : a.P); ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float f[4];
                const unsigned char* q = gr + r * kGrad + h * 128 * sizeof(G);
                if constexpr (GT == ZERO_TYPE_FP32) {
                    *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(q);
                } else {
                    const uint2 u = *reinterpret_cast<const uint2*>(q);
                    const float2 f0 = unpack2<GT>(u.x), f1 = unpack2<GT>(u.y);
                    f[0] = f0.x, f[1] = f0.y, f[2] = f1.x, f[3] = f1.y;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) g[4 * h + j] = ONE ? f[j] : __fadd_rn(g[4 * h + j], f[j]);
            }
        hand_back(s);
        const long long i0 = b0 + lane * 4;
        update<BITS, ONE>(a, k, w, m, v, g, mc, vc,
                          [&](int j) { return static_cast<unsigned int>(i0 >> 1) + (j >> 1) + (j >= 4 ? 62u : 0u); },
                          [](int j) { return (j & 1) != 0; });
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const long long i = i0 + h * 128;
            __stcs(reinterpret_cast<float4*>(ch.w + i), *reinterpret_cast<float4*>(w + 4 * h));
            if constexpr (BITS == 32) {
                __stcs(reinterpret_cast<float4*>(static_cast<float*>(ch.m) + i), *reinterpret_cast<float4*>(m + 4 * h));
                __stcs(reinterpret_cast<float4*>(static_cast<float*>(ch.v) + i), *reinterpret_cast<float4*>(v + 4 * h));
            } else {
                __stcs(reinterpret_cast<unsigned int*>(static_cast<unsigned char*>(ch.m) + i), mc[h]);
                __stcs(reinterpret_cast<unsigned int*>(static_cast<unsigned char*>(ch.v) + i), vc[h]);
            }
            __stcs(reinterpret_cast<uint2*>(static_cast<unsigned short*>(ch.p) + i),
                   make_uint2(pack2<PT>(w[4 * h], w[4 * h + 1]), pack2<PT>(w[4 * h + 2], w[4 * h + 3])));
        }
    }
}

// ---------------------------------------------------------------------------
// The norm
// ---------------------------------------------------------------------------

// Each thread squares eight means at a time and adds their sum to a
// compensated fp32 sum (Kahan): the rounding error does not grow with the
// number of elements.  Eights whose sum is outside [2^-80, 2^100] (below, small
// squares are lost; above, the sums of many may overflow) are squared again
// after scaling and added in fp64.  The CTAs' sums are joined in fp64 by the last CTA to
// finish, in CTA order, so the bits do not depend on which one that is.
// Bound by HBM reads: eight fp16 ranks of 3.0e8 parameters 671 us (7200 GB/s,
// 1.06 of the measured copy bandwidth); 50 thousand parameters 6.3 us.  The
// check of the range costs 0.15 us of those, and 1 % of one bf16 rank's 3.0e8
// (91.7 to 92.8 us; all zeros 97 us, all of 1e-25 153 us).  The branch for
// the others is kept out of the main path's way and spills 10 to 74 bytes.
// Short lists take small chunks, so that every SM has some, and read four
// ranks at once instead of four vectors of one (eight bf16 ranks of 2.4e5
// parameters 11.4 against 8.1 us; long lists lose, 4.0e8 parameters of one rank
// 124 against 233 us).
template <int GT, int VECS>
__global__ void __launch_bounds__(kThreads, 4) zero_grad_norm_kernel(const __grid_constant__ Args a)
{
    using G = typename Elem<GT>::type;
    constexpr int kNormChunk = VECS * kNormStep, kRanks = VECS == 1 ? 4 : 1;
    const int tid = threadIdx.x;
    let_successor_start();
    wait_for_predecessor();
    float sum = 0.0f, comp = 0.0f;
    auto add = [&](float s) {
        const float y = __fsub_rn(s, comp), t = __fadd_rn(sum, y);
        comp = __fsub_rn(__fsub_rn(t, sum), y);
        sum = t;
    };
    double wide = 0.0;
    bool scaled = false; // fp64 operations are few a cycle: not even one more where none is needed
    auto add_scaled = [&](const float (&g)[8], bool low) {
        unsigned int any = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) any |= __float_as_uint(g[j]);
        if ((any & 0x7fffffffu) == 0) return; // zeros
        const float f = low ? 1.2676506002282294e30f : 8.470329472543003e-22f; // 2^100 (means below 2^-40), 2^-70
        float s = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = __fmul_rn(g[j], f);
            s = fmaf(x, x, s);
        }
        wide += static_cast<double>(s) * (low ? 6.223015277861142e-61 : 1.393796574908164e42); // 2^-200, 2^140
        scaled = true;
    };
    long long lo = 0, hi = 0, n = 0, stride = 0;
    int phase = 0;
    const G* gp = nullptr;
    for (long long c = blockIdx.x; c < a.chunks; c += gridDim.x) {
        if (c >= hi) {
            const int ti = find_tensor(a.first, a.n_tensors, c);
            lo = __ldg(a.first + ti);
            hi = __ldg(a.first + ti + 1);
            const Tensor* x = a.tensors + ti;
            n = x->n;
            stride = x->stride;
            phase = x->gphase;
            gp = static_cast<const G*>(x->g);
        }
        const long long c0 = (c - lo) * kNormChunk - max(phase, 0);
        float acc[VECS][8];
#pragma unroll
        for (int k = 0; k < VECS; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[k][j] = 0.0f;
        if (phase >= 0 && c0 >= 0 && c0 + kNormChunk <= n) {
#pragma unroll kRanks
            for (int r = 0; r < a.P; ++r) {
                Raw8<GT> raw[VECS];
#pragma unroll
                for (int k = 0; k < VECS; ++k) raw[k] = load8<GT>(gp + r * stride + c0 + (k * kThreads + tid) * 8);
#pragma unroll
                for (int k = 0; k < VECS; ++k) add8<GT>(acc[k], raw[k]);
            }
        } else { // a tensor's end, or rows off 16 bytes: one element an access, lanes side by side, the loads of a rank together
#pragma unroll kRanks
            for (int r = 0; r < a.P; ++r) {
                const G* row = gp + r * stride + c0 + tid;
#pragma unroll
                for (int k = 0; k < VECS; ++k) {
                    float e[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const long long at = c0 + tid + (k * 8 + j) * kThreads;
                        e[j] = at >= 0 && at < n ? to_float(row[(k * 8 + j) * kThreads]) : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[k][j] = __fadd_rn(acc[k][j], e[j]);
                }
            }
        }
        float s[VECS], low = kHighSquares, high = 0.0f;
#pragma unroll
        for (int k = 0; k < VECS; ++k) {
            s[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc[k][j] = mean_of(acc[k][j], a);
                s[k] = fmaf(acc[k][j], acc[k][j], s[k]);
            }
            low = min_or_nan(low, s[k]);
            high = max_or_nan(high, s[k]);
        }
        if (__builtin_expect(low >= kLowSquares && high <= kHighSquares, 1)) {
#pragma unroll
            for (int k = 0; k < VECS; ++k) add(s[k]);
        } else {
#pragma unroll
            for (int k = 0; k < VECS; ++k) {
                if (s[k] >= kLowSquares && s[k] <= kHighSquares) add(s[k]);
                else add_scaled(acc[k], s[k] < kLowSquares);
            }
        }
    }

    __shared__ double part[kWarps];
    __shared__ bool last;
    auto block_sum = [&](double d) { // in thread 0
        for (int o = 16; o; o >>= 1) d += __shfl_down_sync(0xffffffffu, d, o);
        if ((tid & 31) == 0) part[tid >> 5] = d;
        __syncthreads();
        d = 0.0;
        if (tid == 0)
            for (int k = 0; k < kWarps; ++k) d += part[k];
        return d;
    };
    double mine = static_cast<double>(sum) - static_cast<double>(comp);
    if (scaled) mine += wide;
    mine = block_sum(mine);
    if (tid == 0) {
        a.head->partial[blockIdx.x] = mine;
        __threadfence();
        last = atomicInc(&a.head->ticket, gridDim.x - 1) == gridDim.x - 1; // wraps to 0 for the next call
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double d = 0.0;
    for (int k = tid; k < static_cast<int>(gridDim.x); k += kThreads) d += __ldcg(&a.head->partial[k]);
    __syncthreads(); // part is read above
    d = block_sum(d);
    if (tid == 0) {
        const float norm = static_cast<float>(sqrt(d) * static_cast<double>(a.grad_scale));
        const bool finite = isfinite(norm);
        float clip = 1.0f;
        if (a.max_norm > 0.0f) clip = fminf(1.0f, __fdiv_rn(a.max_norm, __fadd_rn(norm, 1e-6f)));
        a.out[0] = norm;
        a.out[1] = finite ? __fmul_rn(a.grad_scale, clip) : 0.0f;
        a.out[2] = finite ? 1.0f : 0.0f;
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using Kernel = void (*)(Args);

int record(cudaError_t e) { return zero_record_cuda_error(static_cast<int>(e)); }

// CTAs of a kernel that fit the current device at once, asked for once (and
// its shared memory allowed).
int resident_ctas(Kernel fn, int threads, int smem, int* out)
{
    static std::mutex mu;
    static std::vector<std::pair<std::pair<int, Kernel>, int>> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record(e);
    std::lock_guard<std::mutex> lock(mu);
    for (const auto& k : known)
        if (k.first.first == dev && k.first.second == fn) {
            *out = k.second;
            return ZERO_OK;
        }
    int per_sm = 0, sms = 0;
    if (smem) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, fn, threads, static_cast<size_t>(smem));
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return record(e);
    *out = std::max(1, per_sm * sms);
    try {
        known.push_back({{dev, fn}, *out});
    } catch (const std::bad_alloc&) {
    }
    return ZERO_OK;
}

struct StepKernels {
    Kernel vector, pipeline;
};

template <int GT, int PT> StepKernels pick_bits(int bits, bool one)
{
    if (bits == 32)
        return one ? StepKernels{zero_adamw_kernel<GT, PT, 32, true>, zero_adamw_pipeline_kernel<GT, PT, 32, true>}
                   : StepKernels{zero_adamw_kernel<GT, PT, 32, false>, zero_adamw_pipeline_kernel<GT, PT, 32, false>};
    return one ? StepKernels{zero_adamw_kernel<GT, PT, 8, true>, zero_adamw_pipeline_kernel<GT, PT, 8, true>}
               : StepKernels{zero_adamw_kernel<GT, PT, 8, false>, zero_adamw_pipeline_kernel<GT, PT, 8, false>};
}

template <int GT> StepKernels pick_param(int param, int bits, bool one)
{
    return param == ZERO_TYPE_FP16 ? pick_bits<GT, ZERO_TYPE_FP16>(bits, one) : pick_bits<GT, ZERO_TYPE_BF16>(bits, one);
}

StepKernels pick_step(int grad, int param, int bits, int P)
{
    switch (grad) {
    case ZERO_TYPE_FP16: return pick_param<ZERO_TYPE_FP16>(param, bits, P == 1);
    case ZERO_TYPE_BF16: return pick_param<ZERO_TYPE_BF16>(param, bits, P == 1);
    default: return pick_param<ZERO_TYPE_FP32>(param, bits, P == 1);
    }
}

template <int GT> Kernel pick_vecs(int vecs)
{
    return vecs == 1 ? zero_grad_norm_kernel<GT, 1> : zero_grad_norm_kernel<GT, kNormVecs>;
}

Kernel pick_norm(int grad, int vecs)
{
    switch (grad) {
    case ZERO_TYPE_FP16: return pick_vecs<ZERO_TYPE_FP16>(vecs);
    case ZERO_TYPE_BF16: return pick_vecs<ZERO_TYPE_BF16>(vecs);
    default: return pick_vecs<ZERO_TYPE_FP32>(vecs);
    }
}

// Stages of the pipeline: the multiple of the groups nearest to 112 KB, one
// each at least where they fit.
int pipeline_stages(int64_t stage)
{
    const int64_t most = std::min<int64_t>(kMaxStages, kPipeSmem / stage) / kGroups;
    const int64_t near = std::max<int64_t>(1, (2 * kPipeTarget / (stage * kGroups) + 1) / 2);
    return static_cast<int>(std::min(near, most)) * kGroups;
}

// Where the pipeline takes over: one threshold for all, near the crossings and not
// on them.  Measured (GB/s, vector against pipeline): 32-bit moments, P = 1, 3.0e8 elements 6070 / 6640, 1.2e7 5560 /
// 5690, 3.9e6 4920 / 4350; P = 2 6740 / 6660, P = 4 6730 / 6740, P = 8 6640 /
// 6470 (more ranks read more than they write and leave the vector kernel
// enough copies in flight).  8-bit moments, P = 1, 3.0e8 elements 5860 / 6300,
// 9.4e6 4170 / 4080, 3.9e6 3160 / 2730; P = 4 9.4e6 4550 / 5000; P = 8 5.0e7
// 5580 / 6990.  Repeated on one list of bf16, 8 bit, P = 1 (us): 8.4e6 20.4 / 22.5,
// 9.4e6 23.6 / 28.0, 1.6e7 46.1 / 42.6: between 8.4e6 and some 1.3e7 elements the
// vector kernel would be up to a sixth quicker.
bool takes_pipeline(int64_t chunks, int bits, int P) { return chunks >= 4096 && (bits == 8 || P == 1); }

int64_t table_size(int64_t n)
{
    return static_cast<int64_t>(sizeof(Header)) + 2 * (n + 1) * 8 + n * static_cast<int64_t>(sizeof(Tensor));
}

static_assert(sizeof(Header) % 16 == 0 && sizeof(Tensor) % 8 == 0, "table layout");

bool good_plan(const zero_adamw_plan_t* p, const void* table)
{
    return p && table && p->n_tensors >= 1 && p->P >= 1 && p->P <= ZERO_MAX_RANKS && p->grad_type >= 0 &&
           p->grad_type <= 2 && p->elements >= 0 && p->chunks >= 0 && p->norm_chunks >= 0 && (p->norm_vecs == 1 || p->norm_vecs == kNormVecs) &&
           p->table_bytes == table_size(p->n_tensors);
}

Args base_args(const zero_adamw_plan_t* plan, void* table, bool norm)
{
    Args a{};
    unsigned char* t = static_cast<unsigned char*>(table);
    a.head = reinterpret_cast<Header*>(t);
    const long long* first = reinterpret_cast<const long long*>(t + sizeof(Header));
    a.first = norm ? first + plan->n_tensors + 1 : first;
    a.tensors = reinterpret_cast<const Tensor*>(first + 2 * (static_cast<int64_t>(plan->n_tensors) + 1));
    a.n_tensors = plan->n_tensors;
    a.P = plan->P;
    a.p_pow2 = (plan->P & (plan->P - 1)) == 0;
    a.inv_p = 1.0f / static_cast<float>(plan->P);
    a.chunks = norm ? plan->norm_chunks : plan->chunks;
    return a;
}

int launch(Kernel fn, const Args& a, long long most, int threads, int smem, void* stream)
{
    int fit = 0;
    const int rc = resident_ctas(fn, threads, smem, &fit);
    if (rc) return rc;
    const long long ctas = std::max(1ll, std::min(std::min<long long>(fit, most), static_cast<long long>(a.chunks)));
    // the kernel may be set up while its predecessor ends (it waits for it before it reads anything)
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned int>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned int>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, a);
    return e == cudaSuccess ? ZERO_OK : record(e);
}

struct Span {
    uintptr_t at, end;
};

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

// The vector phase of streams that are `size` bytes an element: elements past
// a boundary of 8 elements; fp32 vectors are 4 elements long, so their phase
// only has to agree modulo 4.
bool phase_is(uintptr_t at, int size, int phase)
{
    const int q = size == 4 ? 4 : 8;
    return static_cast<int>((at / size) % q) == phase % q;
}

int plan_tensors(const zero_adamw_tensor_t* tensors, int32_t n_tensors, int32_t P, int32_t grad_type, int32_t bits,
                 zero_adamw_plan_t* plan, unsigned char* table)
{
    const int gs = grad_type == ZERO_TYPE_FP32 ? 4 : 2, ss = bits == 32 ? 4 : 1;
    std::vector<Span> written, read;
    int64_t most = 0; // chunks of the norm of the larger size
    for (int32_t j = 0; j < n_tensors && most <= kShortNorm; ++j) {
        if (tensors[j].n < 0 || tensors[j].n > (INT64_MAX >> 5)) return ZERO_EINVAL;
        most += (tensors[j].n + kNormVecs * kNormStep - 1) / (kNormVecs * kNormStep);
    }
    plan->norm_vecs = most <= kShortNorm ? 1 : kNormVecs;
    const int64_t norm_chunk = static_cast<int64_t>(plan->norm_vecs) * kNormStep;
    long long* first = nullptr;
    Tensor* rec = nullptr;
    if (table) {
        std::memset(table, 0, sizeof(Header));
        first = reinterpret_cast<long long*>(table + sizeof(Header));
        rec = reinterpret_cast<Tensor*>(first + 2 * (static_cast<int64_t>(n_tensors) + 1));
    }
    for (int32_t j = 0; j < n_tensors; ++j) {
        const zero_adamw_tensor_t& t = tensors[j];
        if (t.n < 0 || t.n > (INT64_MAX >> 5)) return ZERO_EINVAL;
        Tensor x{};
        long long chunks = 0, norm_chunks = 0;
        if (bits && (!(t.weight_decay >= 0.0f) || !std::isfinite(t.weight_decay) || !(t.lr_scale >= 0.0f) ||
                     !std::isfinite(t.lr_scale)))
            return ZERO_EINVAL;
        if (t.n > 0) {
            if (!t.grad || (P > 1 && (t.rank_stride < t.n || t.rank_stride > (INT64_MAX >> 14)))) return ZERO_EINVAL;
            const int64_t stride = P > 1 ? t.rank_stride : 0;
            if (addr(t.grad) % gs) return ZERO_EALIGN;
            for (int32_t r = 0; r < P; ++r) {
                const uintptr_t at = addr(t.grad) + static_cast<uintptr_t>(r) * static_cast<uintptr_t>(stride) * gs;
                read.push_back({at, at + static_cast<uintptr_t>(t.n) * gs});
            }
            x.g = t.grad;
            x.stride = stride;
            x.n = t.n;
            x.gphase = static_cast<int>((addr(t.grad) / gs) % 8);
            if ((stride * gs) % 16) x.gphase = -1;
            x.phase = -1;
            if (bits) {
                if (!t.master || !t.m || !t.v || !t.param || (bits == 8 && (!t.m_scale || !t.v_scale)))
                    return ZERO_EINVAL;
                if (addr(t.master) % 4 || addr(t.m) % ss || addr(t.v) % ss || addr(t.param) % 2 ||
                    (bits == 8 && (addr(t.m_scale) % 4 || addr(t.v_scale) % 4)))
                    return ZERO_EALIGN;
                const uintptr_t n = static_cast<uintptr_t>(t.n), blocks = (n + kBlock - 1) / kBlock;
                written.push_back({addr(t.master), addr(t.master) + n * 4});
                written.push_back({addr(t.m), addr(t.m) + n * ss});
                written.push_back({addr(t.v), addr(t.v) + n * ss});
                written.push_back({addr(t.param), addr(t.param) + n * 2});
                if (bits == 8) {
                    written.push_back({addr(t.m_scale), addr(t.m_scale) + blocks * 4});
                    written.push_back({addr(t.v_scale), addr(t.v_scale) + blocks * 4});
                }
                x.w = t.master, x.m = t.m, x.v = t.v, x.ms = t.m_scale, x.vs = t.v_scale, x.p = t.param;
                x.decay = t.weight_decay, x.lr_scale = t.lr_scale;
                // a block of 8-bit scales starts with the tensor, so only phase 0 keeps vectors inside blocks
                const int ph = static_cast<int>((addr(t.param) / 2) % 8);
                if ((bits == 32 || ph == 0) && phase_is(addr(t.grad), gs, ph) && (stride * gs) % 16 == 0 &&
                    phase_is(addr(t.master), 4, ph) && phase_is(addr(t.m), ss, ph) && phase_is(addr(t.v), ss, ph))
                    x.phase = ph;
                // bulk copies start on 16 bytes, which the phase grants all streams but the 8-bit codes
                if (x.phase < 0 || (bits == 8 && (addr(t.m) % 16 || addr(t.v) % 16))) plan->pipeline = 0;
                chunks = (t.n + std::max(x.phase, 0) + kChunk - 1) / kChunk;
                plan->vector_tensors += x.phase >= 0;
            }
            norm_chunks = (t.n + std::max(x.gphase, 0) + norm_chunk - 1) / norm_chunk;
        }
        if (table) {
            first[j] = plan->chunks;
            first[n_tensors + 1 + j] = plan->norm_chunks;
            std::memcpy(rec + j, &x, sizeof(x));
        }
        plan->chunks += chunks;
        plan->norm_chunks += norm_chunks;
        plan->elements += t.n;
    }
    if (table) {
        first[n_tensors] = plan->chunks;
        first[2 * n_tensors + 1] = plan->norm_chunks;
    }
    // no two written spans share a byte, and none shares one with a gradient
    auto by_start = [](const Span& p, const Span& q) { return p.at < q.at; };
    std::sort(written.begin(), written.end(), by_start);
    for (size_t k = 1; k < written.size(); ++k)
        if (written[k].at < written[k - 1].end) return ZERO_EOVERLAP;
    for (const Span& s : read) { // the written spans are disjoint: only the first that ends past s.at can meet it first
        auto it = std::lower_bound(written.begin(), written.end(), s.at,
                                   [](const Span& p, uintptr_t at) { return p.end <= at; });
        if (it != written.end() && it->at < s.end) return ZERO_EOVERLAP;
    }
    return ZERO_OK;
}

} // namespace

extern "C" int zero_adamw_plan(const zero_adamw_tensor_t* tensors, int32_t n_tensors, int32_t P, int32_t grad_type,
                               int32_t param_type, int32_t state_bits, zero_adamw_plan_t* plan, void* table_out,
                               int64_t table_bytes)
{
    if (!tensors || !plan || n_tensors < 1 || P < 1 || P > ZERO_MAX_RANKS || grad_type < 0 || grad_type > 2 ||
        (state_bits != 0 && state_bits != 8 && state_bits != 32) ||
        (state_bits != 0 && param_type != ZERO_TYPE_FP16 && param_type != ZERO_TYPE_BF16))
        return ZERO_EINVAL;
    zero_adamw_plan_t p{};
    p.n_tensors = n_tensors;
    p.P = P;
    p.grad_type = grad_type;
    p.param_type = state_bits ? param_type : ZERO_TYPE_FP16;
    p.state_bits = state_bits;
    p.pipeline = state_bits != 0;
    p.table_bytes = table_size(n_tensors);
    if (table_out && table_bytes < p.table_bytes) return ZERO_EINVAL;
    try {
        // written to a copy first: a refused call leaves the caller's memory as it was
        std::vector<unsigned char> table(table_out ? static_cast<size_t>(p.table_bytes) : 0);
        const int rc = plan_tensors(tensors, n_tensors, P, grad_type, state_bits, &p, table_out ? table.data() : nullptr);
        if (rc) return rc;
        if (table_out) std::memcpy(table_out, table.data(), table.size());
    } catch (const std::bad_alloc&) {
        return ZERO_ENOMEM;
    }
    *plan = p;
    return ZERO_OK;
}

extern "C" int zero_grad_norm(const zero_adamw_plan_t* plan, void* table, float grad_scale, float max_norm,
                              float* stats, void* cuda_stream)
{
    if (!good_plan(plan, table) || !stats || !std::isfinite(grad_scale) || !(grad_scale > 0.0f) ||
        std::isnan(max_norm))
        return ZERO_EINVAL;
    if (addr(table) % 16 || addr(stats) % 4) return ZERO_EALIGN;
    Args a = base_args(plan, table, true);
    a.grad_scale = grad_scale;
    a.max_norm = max_norm;
    a.out = stats;
    return launch(pick_norm(plan->grad_type, plan->norm_vecs), a, kMaxPartials, kThreads, 0, cuda_stream);
}

namespace {

// The arguments of a step, checked.
int step_args(const zero_adamw_plan_t* plan, void* table, const float* stats, int64_t t, float lr, float beta1, float beta2,
              float eps, uint32_t seed, Args* out)
{
    if (!good_plan(plan, table) || (plan->state_bits != 8 && plan->state_bits != 32) || t < 1 ||
        !std::isfinite(lr) || !(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f) ||
        !std::isfinite(eps) || eps < 0.0f || (eps > 0.0f && !std::isnormal(eps)) || // the kernels' reciprocal flushes
        (plan->param_type != ZERO_TYPE_FP16 && plan->param_type != ZERO_TYPE_BF16))
        return ZERO_EINVAL;
    if (addr(table) % 16 || addr(stats) % 4) return ZERO_EALIGN;
    Args& a = *out;
    a = base_args(plan, table, false);
    a.stats = stats;
    a.lr = lr;
    a.b1 = beta1;
    a.b2 = beta2;
    a.omb1 = 1.0f - beta1;
    a.omb2 = 1.0f - beta2;
    a.r1 = static_cast<float>(1.0 / (1.0 - std::pow(static_cast<double>(beta1), static_cast<double>(t))));
    a.c2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(static_cast<double>(beta2), static_cast<double>(t))));
    a.eps = eps;
    a.seed = seed;
    const int64_t stage = kChunk * (4 + plan->state_bits / 4 + (plan->grad_type == ZERO_TYPE_FP32 ? 4 : 2) * int64_t{plan->P});
    a.stages = pipeline_stages(stage);
    a.stage_bytes = static_cast<int>(std::min<int64_t>(stage, kPipeSmem));
    return ZERO_OK;
}

bool step_takes_pipeline(const zero_adamw_plan_t* plan, const Args& a)
{
    return plan->pipeline && a.stages > 0 && takes_pipeline(plan->chunks, plan->state_bits, plan->P);
}

} // namespace

extern "C" int zero_adamw_step(const zero_adamw_plan_t* plan, void* table, const float* stats, int64_t t, float lr,
                               float beta1, float beta2, float eps, uint32_t seed, void* cuda_stream)
{
    Args a{};
    const int rc = step_args(plan, table, stats, t, lr, beta1, beta2, eps, seed, &a);
    if (rc) return rc;
    if (plan->chunks == 0) return ZERO_OK; // no elements
    const StepKernels fn = pick_step(plan->grad_type, plan->param_type, plan->state_bits, plan->P);
    if (step_takes_pipeline(plan, a)) return launch(fn.pipeline, a, INT64_MAX, kPipeThreads, kPipeSmem, cuda_stream);
    return launch(fn.vector, a, INT64_MAX, kThreads, 0, cuda_stream);
}

extern "C" int zero_selftest_adamw_wait(const zero_adamw_plan_t* plan, void* table, int64_t t, float lr, float beta1,
                                        float beta2, float eps, void* cuda_stream)
{
    Args a{};
    int rc = step_args(plan, table, nullptr, t, lr, beta1, beta2, eps, 0, &a);
    if (rc) return rc;
    if (plan->grad_type != ZERO_TYPE_FP16 || plan->param_type != ZERO_TYPE_FP16 || plan->state_bits != 32 || plan->P != 1 ||
        !step_takes_pipeline(plan, a))
        return ZERO_EINVAL;
    const Kernel fn = zero_adamw_pipeline_kernel<ZERO_TYPE_FP16, ZERO_TYPE_FP16, 32, true, true>;
    int ctas = 0;
    if ((rc = resident_ctas(fn, kPipeThreads, kPipeSmem, &ctas))) return rc;
    if (plan->chunks <= int64_t{ctas} * a.stages) return ZERO_EINVAL; // the first CTA must come back to a stage
    return launch(fn, a, INT64_MAX, kPipeThreads, kPipeSmem, cuda_stream);
}

// Bounded waits of the pipeline that gave up (zero_train_timeouts adds them).
__attribute__((visibility("hidden"))) int zero_adamw_wait_timeouts(unsigned int* count, int reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_adamw_timeouts, sizeof(*count));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_adamw_timeouts, &zero, sizeof(zero));
    }
    return e == cudaSuccess ? ZERO_OK : record(e);
}
