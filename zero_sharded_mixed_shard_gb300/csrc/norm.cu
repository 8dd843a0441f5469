// Layer norm over the last axis and its gradients.
//
//   forward   m = mean(x), s = 1 / sqrt(mean((x - m)^2) + eps)
//             y = (x - m) s w + b
//   backward  h = (x - m) s,  a = dy w
//             dx = s (a - mean(a) - h mean(a h)) + r
//             dw = sum over rows of dy h,   db = sum over rows of dy
//
// Both are bound by HBM: a row is read once, held in registers between its
// statistics and its use, and written once, while the rows to come are on their
// way to shared memory.  A group of threads shares a row (eight lanes for
// narrow ones, a CTA for wide ones), each with vectors of 8 elements; the variance is that of the centred values, not a difference of
// large sums, and the centred values' own mean (what rounding left of it) is
// taken out of them: a mean far above the row's spread costs no digits, and a
// constant row's y is the bias.  In the backward pass a thread keeps its columns' sums of dw and
// db over all rows of its group; the groups' sums go to the workspace and a
// second launch adds them in a fixed order, so that a call repeats its bits.
#include "layers.cuh"

namespace {

struct NormArgs {
    const void* x;
    const void* w;
    const void* b;
    void* y;
    float* mean;
    float* rstd;
    long long ldx, ldy, T;
    int D;
    float eps, inv_d;
    float share, whole, inv_whole; // 2^-k, D 2^-k (a half to 1), and one over it
};

struct NormBackArgs {
    const void* dy;
    const void* x;
    const void* w;
    const float* mean;
    const float* rstd;
    const void* res;
    void* dx;
    float* sums;         // [groups][2][D], a part of each CTA, null: no gradients of the weights
    long long lddy, ldx, ldr, lddx, T;
    int D, groups;
    float inv_d;
};

struct NormSumArgs {
    const float* sums;
    void* dw;
    void* db;
    int D, groups, bf16;
};

// A row's columns among the GROUP threads that share it: eight neighbours a
// thread, GROUP threads beside each other, then the next vector of each.
template <int GROUP> __device__ __forceinline__ int column(int k, int self) { return (k * GROUP + self) * 8; }

// VEC: rows lie on 16 bytes and hold whole vectors.  Else they start anywhere.
template <int VEC> __device__ __forceinline__ uint4 load_row(const uint16_t* row, int c, int D)
{
    if constexpr (!VEC) return load_any(row, c, D);
    return c < D ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
}

// By whole warps: lanes of a group that has no row pass D 0.
template <int VEC, int GROUP> __device__ __forceinline__ void store_row(uint16_t* row, int c, int self, int D, const uint4& v)
{
    constexpr int kRun = GROUP < 32 ? GROUP : 32; // lanes beside each other in a row
    if constexpr (!VEC) store_any(row, c, D, v, self % kRun == 0, self % kRun == kRun - 1);
    else if (c < D) *reinterpret_cast<uint4*>(row + c) = v;
}

template <int BF16> __device__ __forceinline__ void widen(const uint4& u, float2 (&v)[4])
{
    v[0] = unpack16(u.x, BF16), v[1] = unpack16(u.y, BF16), v[2] = unpack16(u.z, BF16), v[3] = unpack16(u.w, BF16);
}

template <int BF16> __device__ __forceinline__ void widen(const uint4& u, float (&v)[8])
{
    float2 p[4];
    widen<BF16>(u, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[2 * j] = p[j].x, v[2 * j + 1] = p[j].y;
}

template <int BF16> __device__ __forceinline__ uint4 narrow(const float2 (&v)[4])
{
    return make_uint4(pack16(v[0].x, v[0].y, BF16), pack16(v[1].x, v[1].y, BF16), pack16(v[2].x, v[2].y, BF16), pack16(v[3].x, v[3].y, BF16));
}

// Rows to come, copied to shared memory ahead of their use: AHEAD of them,
// STREAMS matrices, VPT vectors of each of the CTA's threads.  VEC: a thread
// copies what it reads itself, and waits for nobody else.  Else the granules
// that hold a run's columns (a run: the lanes of a warp that share a row) are
// copied by its lanes, one more than there are lanes, and a lane reads two.
template <int VEC, int GROUP, int VPT, int STREAMS, int AHEAD, int THREADS> struct Rows {
    static constexpr int kRun = GROUP < 32 ? GROUP : 32, kSlots = THREADS / kRun * (VEC ? kRun : kRun + 1);
    static constexpr int kBytes = AHEAD * STREAMS * VPT * kSlots * 16;
    uint4* base;
    int self, place; // within the group; of this thread's first granule among kSlots

    __device__ __forceinline__ Rows(unsigned char* raw, int self_) : base(reinterpret_cast<uint4*>(raw)), self(self_)
    {
        place = VEC ? threadIdx.x : threadIdx.x / kRun * (kRun + 1) + threadIdx.x % kRun;
    }
    __device__ __forceinline__ uint4* at(int slot, int stream, int k) { return base + ((slot * STREAMS + stream) * VPT + k) * kSlots + place; }
    static __device__ __forceinline__ void copy16(void* to, const void* from)
    {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
    }
    // Granules that hold no element of the row are not read.
    __device__ __forceinline__ void copy(int slot, int stream, const uint16_t* row, int D)
    {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = column<GROUP>(k, self);
            if constexpr (VEC) {
                if (c < D) copy16(at(slot, stream, k), row + c);
            } else {
                const int e = phase_of(row + c);
                if (c - e < D) copy16(at(slot, stream, k), row + c - e);
                if (self % kRun == kRun - 1 && e && c + 8 - e < D) copy16(at(slot, stream, k) + 1, row + c - e + 8);
            }
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    static __device__ __forceinline__ void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD - 1) : "memory");
        if (!VEC) __syncwarp();
    }
    // Before a slot that has been read is copied to again.
    static __device__ __forceinline__ void read()
    {
        if (!VEC) __syncwarp();
    }
    __device__ __forceinline__ uint4 get(int slot, int stream, int k, const uint16_t* row, int D)
    {
        const uint4* p = at(slot, stream, k);
        const int c = column<GROUP>(k, self);
        if constexpr (VEC) return c < D ? p[0] : make_uint4(0, 0, 0, 0);
        return first_of(shifted(p[0], p[1], phase_of(row + c)), D - c);
    }
};

// Sum over a group of up to a warp.
template <int GROUP> __device__ __forceinline__ float lanes_sum(float v)
{
#pragma unroll
    for (int o = (GROUP < 32 ? GROUP : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <int GROUP, int THREADS> __device__ __forceinline__ void group_barrier(int group)
{
    if constexpr (GROUP == THREADS) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(GROUP) : "memory");
}

// Sums over a group's threads of N values, the same in all of them.  `part`
// has room for two turns: a thread passes the next barrier only when all have
// read this turn's values.
template <int GROUP, int N, int THREADS>
__device__ __forceinline__ void group_sum(float (&v)[N], float (*part)[THREADS / 32][N], int group, int* turn)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<GROUP>(v[i]);
    if constexpr (GROUP > 32) {
        constexpr int kWarps = GROUP / 32;
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) part[*turn][threadIdx.x / 32][i] = v[i];
        group_barrier<GROUP, THREADS>(group);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[i] = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) v[i] += part[*turn][group * kWarps + k][i];
        }
        *turn ^= 1;
    }
}

// Values whose squares leave fp32's range (or do with eps) are scaled by 2^-96.
constexpr float kSmall = 1.262177448353619e-29f, kLarge = 7.922816251426434e28f, kMost = 3.402823466e38f;

// The variance, from the mean square and the mean of values about the mean
// (NaN goes on).
__device__ __forceinline__ float centred(float square, float left)
{
    const float v = fmaf(-left, left, square);
    return v < 0.0f ? 0.0f : v;
}

// x / y from y's rounded reciprocal and the remainder: exact where the
// quotient has a float (a constant row's mean).
__device__ __forceinline__ float quotient(float x, float y, float reciprocal)
{
    const float q = x * reciprocal;
    return fmaf(fmaf(-q, y, x), reciprocal, q);
}

// Forward: a CTA that stays on every SM, as many groups as fit in it, a row per
// group at a time.  A thread has four vectors of a row where it is wide enough:
// fewer threads have less to join.  Its weights and biases stay in its
// registers.  16384 rows of 2048 bf16 elements (134 MB) 24 us, 5600 GB/s (two
// vectors a thread, two CTAs an SM, weights in shared memory 35 us: twice the
// joins; a CTA of 256 threads per row that does not stay 40); off 16 bytes 50 us,
// bound by shifting the granules.  The centred values' mean, joined with their
// squares, costs 0.3 of the 24, a division in place of the reciprocal 0.6 more.
constexpr int kNormThreads = 512;
template <int VPT> constexpr int kForwardAhead = VPT == 4 ? 5 : 8;
template <int VEC, int GROUP, int VPT> using ForwardRows = Rows<VEC, GROUP, VPT, 1, kForwardAhead<VPT>, kNormThreads>;

template <int BF16, int VEC, int GROUP, int VPT>
__global__ void __launch_bounds__(kNormThreads, 1) zero_layernorm_kernel(const __grid_constant__ NormArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    constexpr int kGroups = kNormThreads / GROUP, S = kForwardAhead<VPT>;
    __shared__ float part[2][kNormThreads / 32][1], part2[2][kNormThreads / 32][2];
    const int self = threadIdx.x % GROUP, group = threadIdx.x / GROUP;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* w = static_cast<const uint16_t*>(a.w);
    const uint16_t* b = static_cast<const uint16_t*>(a.b);
    uint16_t* y = static_cast<uint16_t*>(a.y);
    ForwardRows<VEC, GROUP, VPT> rows(raw, self);
    const long long step = static_cast<long long>(gridDim.x) * kGroups;
    // the groups of a warp go round equally often: a group without a row works on none
    constexpr int kTogether = GROUP < 32 ? 32 / GROUP : 1;
    const long long first = static_cast<long long>(blockIdx.x) * kGroups + group, leader = first / kTogether * kTogether;
    auto ahead = [&](int slot, long long r) {
        if (r < a.T) rows.copy(slot, 0, x + r * a.ldx, a.D);
        rows.commit();
    };
    for (int s = 0; s < S - 1; ++s) ahead(s, first + s * step);
    uint4 weight[VPT], bias[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t one = BF16 ? 0x3f803f80u : 0x3c003c00u;
        weight[k] = w ? load_row<VEC>(w, column<GROUP>(k, self), a.D) : make_uint4(one, one, one, one);
        bias[k] = b ? load_row<VEC>(b, column<GROUP>(k, self), a.D) : make_uint4(0, 0, 0, 0);
    }
    int s = 0, turn = 0;
    for (long long lead = leader, r = first; lead < a.T; lead += step, r += step) {
        const int D = r < a.T ? a.D : 0;
        const uint16_t* from = x + r * a.ldx;
        rows.read();
        ahead(s == 0 ? S - 1 : s - 1, r + (S - 1) * step); // into the slot that the last row has left
        rows.wait();
        float2 v[VPT][4];
        // the mean as a sum of x 2^-k, exact, with 2^k the power of two from D on: no partial sum is above the largest value
        float2 total = both(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            widen<BF16>(rows.get(s, 0, k, from, D), v[k]);
#pragma unroll
            for (int j = 0; j < 4; ++j) total = fma2(v[k][j], both(a.share), total);
        }
        float sum[1] = {total.x + total.y};
        group_sum<GROUP, 1, kNormThreads>(sum, part, group, &turn);
        const float mean = quotient(sum[0], a.whole, a.inv_whole);
        // half of the centred values: a difference of two values of bf16's range may pass fp32's; 0 past the row's end
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int there = D - column<GROUP>(k, self);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[k][j] = fma2(v[k][j], both(0.5f), both(-0.5f * mean));
                if (VEC ? there <= 0 : there <= 2 * j) v[k][j].x = 0.0f;
                if (VEC ? there <= 0 : there <= 2 * j + 1) v[k][j].y = 0.0f;
            }
        }
        // the centred values' mean (what the mean's rounding left) and their variance
        auto moments = [&](float scale, float* left, float* variance) {
            float2 all = both(0.0f), one = both(0.0f);
#pragma unroll
            for (int k = 0; k < VPT; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = mul2(v[k][j], both(scale));
                    one = add2(one, d);
                    all = fma2(d, d, all);
                }
            float q[2] = {one.x + one.y, all.x + all.y};
            group_sum<GROUP, 2, kNormThreads>(q, part2, group, &turn);
            *left = q[0] * a.inv_d;
            *variance = centred(q[1] * a.inv_d, *left);
        };
        float left, q;
        moments(1.0f, &left, &q);
        const float spread = fmaf(4.0f, q, a.eps);
        float rstd = __frsqrt_rn(spread);
        // squares of values above 2^63 leave fp32's range: taken again with the values scaled down (by the whole warp where
        // groups share one: the sum's shuffles are the warp's)
        const int over = !(spread <= kMost);
        if (BF16 && (GROUP < 32 ? __any_sync(0xffffffffu, over) : over)) {
            float small_left, small;
            moments(kSmall, &small_left, &small);
            if (over) rstd = __frsqrt_rn(fmaf(4.0f, small, a.eps * kSmall * kSmall)) * kSmall, left = small_left * kLarge;
        }
        const float twice = 2.0f * rstd, back = -left * twice;
        if (self == 0 && D) {
            if (a.mean) a.mean[r] = fmaf(2.0f, left, mean);
            if (a.rstd) a.rstd[r] = rstd;
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = column<GROUP>(k, self);
            float2 g[4], h[4];
            widen<BF16>(weight[k], g);
            widen<BF16>(bias[k], h);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[k][j] = fma2(fma2(v[k][j], both(twice), both(back)), g[j], h[j]);
            store_row<VEC, GROUP>(y + r * a.ldy, c, self, D, narrow<BF16>(v[k]));
        }
        if (++s == S) s = 0;
    }
}

// Forward of rows above 16384 elements: a CTA per row, which reads it three
// times (from L2 after the first).
constexpr int kWideThreads = 1024;

template <int BF16, int VEC>
__global__ void __launch_bounds__(kWideThreads) zero_layernorm_wide_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float part[2][kWideThreads / 32][1], part2[2][kWideThreads / 32][2];
    const int self = threadIdx.x;
    const long long r = blockIdx.x;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + r * a.ldx;
    const uint16_t* w = static_cast<const uint16_t*>(a.w);
    const uint16_t* b = static_cast<const uint16_t*>(a.b);
    uint16_t* y = static_cast<uint16_t*>(a.y) + r * a.ldy;
    const int steps = (a.D + kWideThreads * 8 - 1) / (kWideThreads * 8);
    int turn = 0;
    float sum[1] = {0.0f};
#pragma unroll 2
    for (int k = 0; k < steps; ++k) {
        float v[8];
        widen<BF16>(load_row<VEC>(x, column<kWideThreads>(k, self), a.D), v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[j], a.share, sum[0]);
    }
    group_sum<kWideThreads, 1, kWideThreads>(sum, part, 0, &turn);
    const float mean = sum[0] / a.whole, half_mean = -0.5f * mean;
    auto moments = [&](float scale, float* left, float* variance) {
        float q[2] = {0.0f, 0.0f};
#pragma unroll 2
        for (int k = 0; k < steps; ++k) {
            float v[8];
            const int c = column<kWideThreads>(k, self);
            widen<BF16>(load_row<VEC>(x, c, a.D), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float d = fmaf(v[j], 0.5f, half_mean) * scale;
                if (c + j < a.D) {
                    q[0] += d;
                    q[1] = fmaf(d, d, q[1]);
                }
            }
        }
        group_sum<kWideThreads, 2, kWideThreads>(q, part2, 0, &turn);
        *left = q[0] * a.inv_d;
        *variance = centred(q[1] * a.inv_d, *left);
    };
    float left, q;
    moments(1.0f, &left, &q);
    const float spread = fmaf(4.0f, q, a.eps);
    float rstd = __frsqrt_rn(spread);
    if (BF16 && !(spread <= kMost)) { // the same in every thread
        float small_left, small;
        moments(kSmall, &small_left, &small);
        rstd = __frsqrt_rn(fmaf(4.0f, small, a.eps * kSmall * kSmall)) * kSmall, left = small_left * kLarge;
    }
    if (self == 0) {
        if (a.mean) a.mean[r] = fmaf(2.0f, left, mean);
        if (a.rstd) a.rstd[r] = rstd;
    }
    const float twice = 2.0f * rstd, back = -left * twice;
    for (int k = 0; k < steps; ++k) {
        const int c = column<kWideThreads>(k, self);
        float v[8], g[8], h[8];
        widen<BF16>(load_row<VEC>(x, c, a.D), v);
        if (w) widen<BF16>(load_row<VEC>(w, c, a.D), g);
        if (b) widen<BF16>(load_row<VEC>(b, c, a.D), h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = fmaf(fmaf(v[j], 0.5f, half_mean), twice, back);
            if (w) v[j] *= g[j];
            if (b) v[j] += h[j];
        }
        store_row<VEC, kWideThreads>(y, c, self, a.D, pack8(v, BF16));
    }
}

// The gradient: a CTA of kGradThreads on every SM, as many groups as fit in it,
// a row per group at a time.  A group joins its two sums of a row by one
// barrier of its own.  16384 rows of 2048 bf16 elements with the residual (269
// MB) 46 us with the sums' launch, 5850 GB/s (rows read where they are used,
// the CTA's barrier twice per four rows: 81 us); off 16 bytes 71 us.  Above 12288
// columns the columns' sums fill the registers: 40 to 264 bytes spilled, one row
// ahead (2048 x 16384 69 us, off 16 bytes 113).
constexpr int kGradThreads = 512;
template <int VPT> constexpr int kGradAhead = VPT == 1 ? 6 : VPT == 2 ? 4 : 2;
template <int VEC, int GROUP, int VPT> using GradRows = Rows<VEC, GROUP, VPT, 3, kGradAhead<VPT>, kGradThreads>;
constexpr int kGradSums = 2 * kGradThreads * 8 * 4; // bytes of the groups' sums, for each vector of a thread

template <int BF16, int VEC, int GROUP, int VPT>
__global__ void __launch_bounds__(kGradThreads, 1) zero_layernorm_grad_kernel(const __grid_constant__ NormBackArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    constexpr int kGroups = kGradThreads / GROUP, S = kGradAhead<VPT>;
    __shared__ float part[2][kGradThreads / 32][2];
    const int self = threadIdx.x % GROUP, group = threadIdx.x / GROUP;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* res = static_cast<const uint16_t*>(a.res);
    uint16_t* dx = static_cast<uint16_t*>(a.dx);
    float2 dw[VPT][4], db[VPT][4];
    uint4 w[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const uint32_t one = BF16 ? 0x3f803f80u : 0x3c003c00u;
        w[k] = a.w ? load_row<VEC>(static_cast<const uint16_t*>(a.w), column<GROUP>(k, self), a.D) : make_uint4(one, one, one, one);
#pragma unroll
        for (int j = 0; j < 4; ++j) dw[k][j] = db[k][j] = both(0.0f);
    }
    GradRows<VEC, GROUP, VPT> rows(raw, self);
    const long long step = static_cast<long long>(gridDim.x) * kGroups;
    constexpr int kTogether = GROUP < 32 ? 32 / GROUP : 1;
    const long long first = static_cast<long long>(blockIdx.x) * kGroups + group, leader = first / kTogether * kTogether;
    auto ahead = [&](int slot, long long r) {
        if (r < a.T) {
            rows.copy(slot, 0, x + r * a.ldx, a.D);
            rows.copy(slot, 1, dy + r * a.lddy, a.D);
            if (res) rows.copy(slot, 2, res + r * a.ldr, a.D);
        }
        rows.commit();
    };
    float mean_next = 0.0f, rstd_next = 0.0f;
    if (first < a.T) mean_next = a.mean[first], rstd_next = a.rstd[first];
    for (int s = 0; s < S - 1; ++s) ahead(s, first + s * step);
    int s = 0, turn = 0;
    for (long long lead = leader, r = first; lead < a.T; lead += step, r += step) {
        const int D = r < a.T ? a.D : 0; // a group without a row works on none
        const float mean = -0.5f * mean_next, rstd = 2.0f * rstd_next;
        if (r + step < a.T) mean_next = a.mean[r + step], rstd_next = a.rstd[r + step];
        rows.read();
        ahead(s == 0 ? S - 1 : s - 1, r + (S - 1) * step); // into the slot that the last row has left
        rows.wait();
        // the row's vectors; more than two of a thread are read again after the joins, its registers hold the columns' sums
        constexpr bool kHeld = VPT < 3;
        uint4 px[VPT], pd[VPT];
        auto get = [&](int k) {
            px[k] = rows.get(s, 0, k, x + r * a.ldx, D);
            pd[k] = rows.get(s, 1, k, dy + r * a.lddy, D);
        };
        if (kHeld)
#pragma unroll
            for (int k = 0; k < VPT; ++k) get(k);
        float2 sum_g = both(0.0f), sum_gh = both(0.0f);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float2 vx[4], vd[4], vw[4];
            if (!kHeld) get(k);
            widen<BF16>(px[k], vx);
            widen<BF16>(pd[k], vd);
            widen<BF16>(w[k], vw);
            // past the row's end dy is 0: such sums go nowhere, so long as their h is finite
            const int there = D - column<GROUP>(k, self);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 h = mul2(fma2(vx[j], both(0.5f), both(mean)), both(rstd));
                if (VEC ? there <= 0 : there <= 2 * j) h.x = 0.0f;
                if (VEC ? there <= 0 : there <= 2 * j + 1) h.y = 0.0f;
                const float2 g = mul2(vd[j], vw[j]);
                dw[k][j] = fma2(vd[j], h, dw[k][j]);
                db[k][j] = add2(db[k][j], vd[j]);
                sum_g = add2(sum_g, g);
                sum_gh = fma2(g, h, sum_gh);
            }
        }
        if (dx) {
            float sum[2] = {sum_g.x + sum_g.y, sum_gh.x + sum_gh.y};
            group_sum<GROUP, 2, kGradThreads>(sum, part, group, &turn);
            const float c0 = sum[0] * a.inv_d, c1 = sum[1] * a.inv_d, half = 0.5f * rstd;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float2 vx[4], vd[4], vw[4], o[4];
                if (!kHeld) get(k);
                widen<BF16>(px[k], vx);
                widen<BF16>(pd[k], vd);
                widen<BF16>(w[k], vw);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = both(0.0f);
                if (res) widen<BF16>(rows.get(s, 2, k, res + r * a.ldr, D), o);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 h = mul2(fma2(vx[j], both(0.5f), both(mean)), both(rstd));
                    const float2 t = add2(fma2(vd[j], vw[j], both(-c0)), mul2(h, both(-c1)));
                    o[j] = fma2(t, both(half), o[j]);
                }
                store_row<VEC, GROUP>(dx + r * a.lddx, column<GROUP>(k, self), self, D, narrow<BF16>(o));
            }
        }
        if (++s == S) s = 0;
    }
    if (!a.sums) return;
    // the groups' sums, joined in the groups' order
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* all = reinterpret_cast<float*>(raw); // [kGroups][2][8 GROUP VPT]
    constexpr int kWidth = 8 * GROUP * VPT;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = column<GROUP>(k, self) + 2 * j;
            *reinterpret_cast<float2*>(all + (group * 2) * kWidth + c) = dw[k][j];
            *reinterpret_cast<float2*>(all + (group * 2 + 1) * kWidth + c) = db[k][j];
        }
    }
    __syncthreads();
    float* to = a.sums + static_cast<long long>(blockIdx.x) * 2 * a.D;
    for (int i = threadIdx.x; i < 2 * kWidth; i += kGradThreads) {
        const int which = i / kWidth, c = i - which * kWidth;
        if (c >= a.D) continue;
        float v = 0.0f;
#pragma unroll 8
        for (int k = 0; k < kGroups; ++k) v += all[(k * 2 + which) * kWidth + c];
        to[which * static_cast<long long>(a.D) + c] = v;
    }
}

// Rows of more than 16384 elements: dx with a CTA per row that reads it twice
// (the second time from L2), the sums of dw and db by stripes of columns.
template <int BF16, int VEC>
__global__ void __launch_bounds__(kWideThreads) zero_layernorm_wide_grad_kernel(const __grid_constant__ NormBackArgs a)
{
    __shared__ float part[2][kWideThreads / 32][2];
    const int self = threadIdx.x;
    const long long r = blockIdx.x;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + r * a.lddy;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + r * a.ldx;
    const uint16_t* w = static_cast<const uint16_t*>(a.w);
    const uint16_t* res = static_cast<const uint16_t*>(a.res) + (a.res ? r * a.ldr : 0);
    uint16_t* dx = static_cast<uint16_t*>(a.dx) + r * a.lddx;
    const float mean = -0.5f * a.mean[r], rstd = 2.0f * a.rstd[r];
    const int steps = (a.D + kWideThreads * 8 - 1) / (kWideThreads * 8);
    int turn = 0;
    float sum[2] = {0.0f, 0.0f};
#pragma unroll 2
    for (int k = 0; k < steps; ++k) {
        float vx[8], vd[8], vw[8];
        const int c = column<kWideThreads>(k, self);
        widen<BF16>(load_row<VEC>(x, c, a.D), vx);
        widen<BF16>(load_row<VEC>(dy, c, a.D), vd);
        if (w) widen<BF16>(load_row<VEC>(w, c, a.D), vw);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (c + j < a.D) {
                const float g = w ? vd[j] * vw[j] : vd[j];
                sum[0] += g;
                sum[1] = fmaf(g, fmaf(vx[j], 0.5f, mean) * rstd, sum[1]);
            }
        }
    }
    group_sum<kWideThreads, 2, kWideThreads>(sum, part, 0, &turn);
    const float c0 = sum[0] * a.inv_d, c1 = sum[1] * a.inv_d, s = 0.5f * rstd;
    for (int k = 0; k < steps; ++k) {
        float vx[8], vd[8], vw[8], o[8];
        const int c = column<kWideThreads>(k, self);
        widen<BF16>(load_row<VEC>(x, c, a.D), vx);
        widen<BF16>(load_row<VEC>(dy, c, a.D), vd);
        if (w) widen<BF16>(load_row<VEC>(w, c, a.D), vw);
        if (a.res) widen<BF16>(load_row<VEC>(res, c, a.D), o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = w ? vd[j] * vw[j] : vd[j], h = fmaf(vx[j], 0.5f, mean) * rstd;
            const float d = s * (g - c0 - h * c1);
            o[j] = a.res ? o[j] + d : d;
        }
        store_row<VEC, kWideThreads>(dx, c, self, a.D, pack8(o, BF16));
    }
}

constexpr int kNormStripe = 256; // columns of a CTA: 32 lanes of 8, for 8 rows at a time

template <int BF16, int VEC>
__global__ void __launch_bounds__(256) zero_layernorm_columns_kernel(const __grid_constant__ NormBackArgs a)
{
    __shared__ float part[2][8][kNormStripe];
    const int lane = threadIdx.x & 31, line = threadIdx.x >> 5;
    const int c0 = static_cast<int>(blockIdx.x / a.groups) * kNormStripe, cols = min(kNormStripe, a.D - c0);
    const int group = static_cast<int>(blockIdx.x % a.groups);
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy) + c0;
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + c0;
    const long long r0 = a.T * group / a.groups, r1 = a.T * (group + 1) / a.groups;
    float dw[8], db[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
#pragma unroll 4
    for (long long r = r0 + line; r < r1; r += 8) {
        float vx[8], vd[8];
        widen<BF16>(load_row<VEC>(x + r * a.ldx, lane * 8, cols), vx);
        widen<BF16>(load_row<VEC>(dy + r * a.lddy, lane * 8, cols), vd);
        const float mean = -0.5f * a.mean[r], rstd = 2.0f * a.rstd[r];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = fmaf(vd[j], fmaf(vx[j], 0.5f, mean) * rstd, dw[j]);
            db[j] += vd[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        part[0][line][lane * 8 + j] = dw[j];
        part[1][line][lane * 8 + j] = db[j];
    }
    __syncthreads();
    const int c = threadIdx.x;
    if (c >= cols) return;
    float sw = 0.0f, sb = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        sw += part[0][k][c];
        sb += part[1][k][c];
    }
    float* to = a.sums + static_cast<long long>(group) * 2 * a.D + c0 + c;
    to[0] = sw;
    to[a.D] = sb;
}

// The groups' sums of a column, in a fixed order: 32 threads of a CTA take
// every 32nd group each, then a warp adds theirs.
__global__ void __launch_bounds__(1024) zero_layernorm_sum_kernel(const __grid_constant__ NormSumArgs a)
{
    __shared__ float part[32][33];
    const int lane = threadIdx.x & 31, line = threadIdx.x >> 5;
    const int stripes = (a.D + 31) / 32;
    const int which = static_cast<int>(blockIdx.x) / stripes, c0 = (static_cast<int>(blockIdx.x) - which * stripes) * 32;
    let_successor_start();
    wait_for_predecessor();
    float s = 0.0f;
    if (c0 + lane < a.D) {
        const float* from = a.sums + static_cast<long long>(which) * a.D + c0 + lane;
#pragma unroll 8
        for (int k = line; k < a.groups; k += 32) s += from[static_cast<long long>(k) * 2 * a.D];
    }
    part[line][lane] = s;
    __syncthreads();
    s = part[lane][line]; // a warp per column now: lane k has the sum of line k
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    void* out = which ? a.db : a.dw;
    if (lane == 0 && c0 + line < a.D && out) store16(out, c0 + line, s, a.bf16);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using NormKernel = void (*)(NormArgs);
using NormBackKernel = void (*)(NormBackArgs);

struct NormPick {
    NormKernel fn;
    int group, smem;     // threads that share a row, bytes of shared memory
};

template <int BF16, int VEC, int GROUP, int VPT> NormPick norm_pick()
{
    return {zero_layernorm_kernel<BF16, VEC, GROUP, VPT>, GROUP, ForwardRows<VEC, GROUP, VPT>::kBytes};
}

template <int BF16, int VEC> NormPick pick_norm(int64_t D)
{
    if (D <= 64) return norm_pick<BF16, VEC, 8, 1>();
    if (D <= 128) return norm_pick<BF16, VEC, 8, 2>();
    if (D <= 256) return norm_pick<BF16, VEC, 8, 4>();
    if (D <= 512) return norm_pick<BF16, VEC, 16, 4>();
    if (D <= 1024) return norm_pick<BF16, VEC, 32, 4>();
    if (D <= 2048) return norm_pick<BF16, VEC, 64, 4>();
    if (D <= 4096) return norm_pick<BF16, VEC, 128, 4>();
    if (D <= 8192) return norm_pick<BF16, VEC, 256, 4>();
    return norm_pick<BF16, VEC, 512, 4>();
}

NormPick pick_norm(int64_t D, int bf16, int vec)
{
    if (bf16) return vec ? pick_norm<1, 1>(D) : pick_norm<1, 0>(D);
    return vec ? pick_norm<0, 1>(D) : pick_norm<0, 0>(D);
}

constexpr int64_t kNormWide = 16384; // rows above it take the wide kernels

struct NormBackPick {
    NormBackKernel fn;
    int group, smem;     // threads that share a row, bytes of shared memory
};

template <int BF16, int VEC, int GROUP, int VPT> NormBackPick back_pick()
{
    return {zero_layernorm_grad_kernel<BF16, VEC, GROUP, VPT>, GROUP, std::max(GradRows<VEC, GROUP, VPT>::kBytes, VPT * kGradSums)};
}

template <int BF16, int VEC> NormBackPick pick_back(int64_t D)
{
    if (D <= 64) return back_pick<BF16, VEC, 8, 1>();
    if (D <= 256) return back_pick<BF16, VEC, 32, 1>();
    if (D <= 512) return back_pick<BF16, VEC, 64, 1>();
    if (D <= 1024) return back_pick<BF16, VEC, 128, 1>();
    if (D <= 2048) return back_pick<BF16, VEC, 128, 2>();
    if (D <= 4096) return back_pick<BF16, VEC, 256, 2>();
    if (D <= 8192) return back_pick<BF16, VEC, 512, 2>();
    if (D <= 12288) return back_pick<BF16, VEC, 512, 3>();
    return back_pick<BF16, VEC, 512, 4>();
}

NormBackPick pick_back(int64_t D, int bf16, int vec)
{
    if (bf16) return vec ? pick_back<1, 1>(D) : pick_back<1, 0>(D);
    return vec ? pick_back<0, 1>(D) : pick_back<0, 0>(D);
}

constexpr int kMostNormCtas = 192; // of the gradient: one on each SM

// Parts of the columns' sums that a gradient's second launch adds, a bound that holds on any device.
int64_t most_groups(int64_t T, int64_t D)
{
    if (D > kNormWide) return std::max<int64_t>(1, std::min<int64_t>(64, T / 64));
    return std::min<int64_t>(kMostNormCtas, T);
}

constexpr int64_t kMostWidth = int64_t{1} << 30; // columns are counted in 32 bits, past the last one too

bool bad_norm(int64_t T, int64_t D, int32_t type)
{
    return T < 0 || T > kMostExtent || D < 1 || D > kMostWidth || T * D > kMostElements ||
           (type != ZERO_TYPE_FP16 && type != ZERO_TYPE_BF16);
}

// Whether n floats at p share a byte with a 16-bit matrix.
bool floats_share(const float* p, int64_t n, const void* q, int64_t ld, int64_t rows, int64_t cols)
{
    return share(p, 2 * n, 1, 2 * n, q, ld, rows, cols);
}

} // namespace

extern "C" int zero_layernorm_forward(const void* x, int64_t ldx, const void* weight, const void* bias, void* y, int64_t ldy,
                                      float* mean, float* rstd, int64_t T, int64_t D, float eps, int32_t type, void* cuda_stream)
{
    if (bad_norm(T, D, type) || !(eps >= 1.17549435e-38f && eps <= 3.4e38f)) return ZERO_EINVAL;
    if (T == 0) return ZERO_OK;
    if (!x || !y || bad_ld(ldx, D) || bad_ld(ldy, D)) return ZERO_EINVAL;
    for (const void* p : {x, weight, bias, static_cast<const void*>(y)})
        if (addr(p) % 2) return ZERO_EALIGN;
    if (addr(mean) % 4 || addr(rstd) % 4) return ZERO_EALIGN;
    const bool same = x == y && ldx == ldy; // in place: a row is read before it is written
    if ((!same && share(y, ldy, T, D, x, ldx, T, D)) || share(y, ldy, T, D, weight, D, 1, D) || share(y, ldy, T, D, bias, D, 1, D) ||
        share(mean, 2 * T, 1, 2 * T, rstd, 2 * T, 1, 2 * T))
        return ZERO_EOVERLAP;
    for (const float* s : {mean, rstd})
        if (floats_share(s, T, x, ldx, T, D) || floats_share(s, T, weight, D, 1, D) || floats_share(s, T, bias, D, 1, D) ||
            floats_share(s, T, y, ldy, T, D))
            return ZERO_EOVERLAP;
    const bool vec = D % 8 == 0 && aligned16(x, ldx) && aligned16(y, ldy) && addr(weight) % 16 == 0 && addr(bias) % 16 == 0;
    const int bf16 = type == ZERO_TYPE_BF16;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    NormArgs a{};
    a.x = x, a.w = weight, a.b = bias, a.y = y, a.mean = mean, a.rstd = rstd, a.ldx = ldx, a.ldy = ldy, a.T = T;
    a.D = static_cast<int>(D), a.eps = eps, a.inv_d = 1.0f / static_cast<float>(D);
    a.share = 1.0f;
    for (int64_t power = 1; power < D; power *= 2) a.share *= 0.5f;
    a.whole = static_cast<float>(D) * a.share, a.inv_whole = 1.0f / a.whole;
    if (D > kNormWide) {
        NormKernel fn;
        if (bf16) fn = vec ? zero_layernorm_wide_kernel<1, 1> : zero_layernorm_wide_kernel<1, 0>;
        else fn = vec ? zero_layernorm_wide_kernel<0, 1> : zero_layernorm_wide_kernel<0, 0>;
        return launch_after(fn, a, T, kWideThreads, 0, 1, st);
    }
    int sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    const NormPick k = pick_norm(D, bf16, vec);
    const int64_t per_cta = kNormThreads / k.group, ctas = std::min<int64_t>((T + per_cta - 1) / per_cta, sms);
    if ((rc = allow_smem(reinterpret_cast<const void*>(k.fn), k.smem))) return rc;
    return launch_after(k.fn, a, ctas, kNormThreads, k.smem, 1, st);
}

extern "C" int zero_layernorm_workspace(int64_t T, int64_t D, int64_t* bytes)
{
    if (!bytes || bad_norm(T, D, ZERO_TYPE_FP16)) return ZERO_EINVAL;
    *bytes = T == 0 ? 0 : up(most_groups(T, D) * 2 * D * 4, 256);
    return ZERO_OK;
}

extern "C" int zero_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                                       const float* mean, const float* rstd, const void* dres, int64_t lddr, void* dx,
                                       int64_t lddx, void* dweight, void* dbias, int64_t T, int64_t D, int32_t type,
                                       void* workspace, int64_t workspace_bytes, void* cuda_stream)
{
    if (bad_norm(T, D, type) || (!dx && !dweight && !dbias)) return ZERO_EINVAL;
    if (!dx) dres = nullptr;
    if (T > 0 && (!dy || !x || !mean || !rstd || bad_ld(lddy, D) || bad_ld(ldx, D) || (dx && bad_ld(lddx, D)) || (dres && bad_ld(lddr, D))))
        return ZERO_EINVAL;
    for (const void* p : {dy, x, weight, dres, static_cast<const void*>(dx), static_cast<const void*>(dweight), static_cast<const void*>(dbias)})
        if (addr(p) % 2) return ZERO_EALIGN;
    if (addr(mean) % 4 || addr(rstd) % 4) return ZERO_EALIGN;
    struct { const void* p; int64_t ld, rows, cols; } out[3] = {{dx, lddx, T, D}, {dweight, D, 1, D}, {dbias, D, 1, D}},
        in[6] = {{dy, lddy, T, D}, {x, ldx, T, D}, {weight, D, 1, D}, {dres, lddr, T, D}, {mean, 2 * T, 1, 2 * T}, {rstd, 2 * T, 1, 2 * T}};
    if (T == 0)
        for (auto& q : in) q.rows = 0;
    for (int i = 0; i < 3; ++i) {
        for (const auto& q : in) {
            // dx over dy or dres: a row is read before it is written; the wide kernels read dy once more
            const bool in_place = i == 0 && q.p == dx && q.ld == lddx && (&q == &in[3] || (&q == &in[0] && D <= kNormWide));
            if (!in_place && share(out[i].p, out[i].ld, out[i].rows, out[i].cols, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
        }
        for (int j = i + 1; j < 3; ++j)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, out[j].p, out[j].ld, out[j].rows, out[j].cols)) return ZERO_EOVERLAP;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (T == 0) { // sums over no rows
        cudaError_t e = cudaSuccess;
        if (dweight) e = cudaMemsetAsync(dweight, 0, static_cast<size_t>(D) * 2, st);
        if (dbias && e == cudaSuccess) e = cudaMemsetAsync(dbias, 0, static_cast<size_t>(D) * 2, st);
        return record(e);
    }
    const bool sums = dweight || dbias;
    if (sums) {
        const int64_t used = up(most_groups(T, D) * 2 * D * 4, 256);
        if (!workspace || workspace_bytes < used) return ZERO_EINVAL;
        if (addr(workspace) % 16) return ZERO_EALIGN;
        for (const auto& q : in)
            if (in_workspace(workspace, used, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
        for (const auto& q : out)
            if (in_workspace(workspace, used, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
    }
    int sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    const int bf16 = type == ZERO_TYPE_BF16;
    const bool vec = D % 8 == 0 && aligned16(dy, lddy) && aligned16(x, ldx) && addr(weight) % 16 == 0 && (!dres || aligned16(dres, lddr)) &&
                     (!dx || aligned16(dx, lddx));
    NormBackArgs a{};
    a.dy = dy, a.x = x, a.w = weight, a.mean = mean, a.rstd = rstd, a.res = dres, a.dx = dx;
    a.sums = sums ? static_cast<float*>(workspace) : nullptr;
    a.lddy = lddy, a.ldx = ldx, a.ldr = lddr, a.lddx = lddx, a.T = T, a.D = static_cast<int>(D), a.inv_d = 1.0f / static_cast<float>(D);
    if (D > kNormWide) {
        a.groups = static_cast<int>(most_groups(T, D));
        NormBackKernel rows, columns;
        if (bf16) rows = vec ? zero_layernorm_wide_grad_kernel<1, 1> : zero_layernorm_wide_grad_kernel<1, 0>;
        else rows = vec ? zero_layernorm_wide_grad_kernel<0, 1> : zero_layernorm_wide_grad_kernel<0, 0>;
        if (bf16) columns = vec ? zero_layernorm_columns_kernel<1, 1> : zero_layernorm_columns_kernel<1, 0>;
        else columns = vec ? zero_layernorm_columns_kernel<0, 1> : zero_layernorm_columns_kernel<0, 0>;
        const int64_t stripes = (D + kNormStripe - 1) / kNormStripe;
        if (stripes * a.groups > INT32_MAX) return ZERO_EINVAL;
        if (dx && (rc = launch_after(rows, a, T, kWideThreads, 0, 1, st))) return rc;
        if (sums && (rc = launch_after(columns, a, stripes * a.groups, 256, 0, 1, st))) return rc;
    } else {
        const NormBackPick k = pick_back(D, bf16, vec);
        const int64_t per_cta = kGradThreads / k.group, ctas = std::min<int64_t>({(T + per_cta - 1) / per_cta, sms, kMostNormCtas});
        a.groups = static_cast<int>(ctas);
        if ((rc = allow_smem(reinterpret_cast<const void*>(k.fn), k.smem))) return rc;
        if ((rc = launch_after(k.fn, a, ctas, kGradThreads, k.smem, 1, st))) return rc;
    }
    if (!sums) return ZERO_OK;
    NormSumArgs s{};
    s.sums = a.sums, s.dw = dweight, s.db = dbias, s.D = a.D, s.groups = a.groups, s.bf16 = bf16;
    const int64_t stripes = (D + 31) / 32;
    return launch_after(zero_layernorm_sum_kernel, s, 2 * stripes, 1024, 0, 1, st);
}
