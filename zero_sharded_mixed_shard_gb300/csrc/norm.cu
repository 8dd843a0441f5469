// Layer norm over the last axis and its gradients.
//
//   forward   m = mean(x), s = 1 / sqrt(mean((x - m)^2) + eps)
//             y = (x - m) s w + b
//   backward  h = (x - m) s,  a = dy w
//             dx = s (a - mean(a) - h mean(a h)) + r
//             dw = sum over rows of dy h,   db = sum over rows of dy
//
// Both are bound by HBM: a row is read once, held in registers between its
// statistics and its use, and written once.  A group of threads shares a row
// (a warp for narrow ones, a CTA for wide ones), each with vectors of 8
// elements; the variance is that of the centred values, not a difference of
// large sums.  In the backward pass a thread keeps its columns' sums of dw and
// db over all rows of its group; the groups' sums go to the workspace and a
// second launch adds them in a fixed order, so that a call repeats its bits.
#include "layers.cuh"

namespace {

constexpr int kNormThreads = 256; // of a CTA, unless a row takes more

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

// Eight elements of a row as they are held between two uses.
struct Packed {
    uint32_t u[4];
};

// Column j of a thread's vector k: 8 neighbours where rows lie on 16 bytes,
// else elements a group's width apart, so that a warp's accesses stay next to
// each other.
template <int VEC, int GROUP> __device__ __forceinline__ int column(int k, int j, int self)
{
    return VEC ? (k * GROUP + self) * 8 + j : (k * 8 + j) * GROUP + self;
}

template <int VEC, int GROUP>
__device__ __forceinline__ Packed load_row(const uint16_t* row, int k, int self, int D)
{
    Packed p;
    if constexpr (VEC) {
        const int c = column<1, GROUP>(k, 0, self);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < D) v = *reinterpret_cast<const uint4*>(row + c);
        p.u[0] = v.x, p.u[1] = v.y, p.u[2] = v.z, p.u[3] = v.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c0 = column<0, GROUP>(k, 2 * j, self), c1 = column<0, GROUP>(k, 2 * j + 1, self);
            const uint32_t lo = c0 < D ? row[c0] : 0, hi = c1 < D ? row[c1] : 0;
            p.u[j] = lo | hi << 16;
        }
    }
    return p;
}

template <int VEC, int GROUP, int BF16>
__device__ __forceinline__ void store_row(uint16_t* row, int k, int self, int D, const float (&v)[8])
{
    if constexpr (VEC) {
        const int c = column<1, GROUP>(k, 0, self);
        if (c < D) *reinterpret_cast<uint4*>(row + c) = pack8(v, BF16);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column<0, GROUP>(k, j, self);
            if (c < D) store16(row, c, v[j], BF16);
        }
    }
}

template <int BF16> __device__ __forceinline__ void widen(const Packed& p, float (&v)[8])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(p.u[j], BF16);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}

// Sums over a group's threads of N values, the same in every thread.  `part`
// has N floats for each of the group's warps; the barriers are the whole CTA's,
// so every thread of it calls this the same number of times.
template <int GROUP, int N> __device__ __forceinline__ void group_sum(float (&v)[N], float* part)
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
    if constexpr (GROUP > 32) {
        constexpr int kWarps = GROUP / 32;
        const int warp = threadIdx.x / 32, lane = threadIdx.x & 31, first = warp / kWarps * kWarps;
        __syncthreads(); // the last call's values have been read
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) part[warp * N + i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) s += part[(first + k) * N + i];
            v[i] = s;
        }
    }
}

template <int GROUP> constexpr int kNormCta = GROUP > kNormThreads ? GROUP : kNormThreads;

// One row per group of GROUP threads, VPT vectors of 8 a thread (D <= 8 GROUP
// VPT).  HELD 0: wider rows, read again for each of the three passes (from L2).
template <int BF16, int VEC, int GROUP, int VPT, int HELD>
__global__ void __launch_bounds__(kNormCta<GROUP>) zero_layernorm_kernel(const __grid_constant__ NormArgs a)
{
    __shared__ float part[kNormCta<GROUP> / 32];
    constexpr int kGroups = kNormCta<GROUP> / GROUP;
    const int self = threadIdx.x % GROUP;
    const long long t = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / GROUP;
    const bool live = t < a.T; // a group without a row goes through the barriers with the others
    const long long row = live ? t : a.T - 1;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* x = static_cast<const uint16_t*>(a.x) + row * a.ldx;
    const int steps = HELD ? 1 : (a.D + GROUP * 8 * VPT - 1) / (GROUP * 8 * VPT);
    Packed p[VPT];
    auto fetch = [&](int s) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) p[k] = load_row<VEC, GROUP>(x, s * VPT + k, self, a.D);
    };
    // the mean as a sum of x / D: no partial sum is above the largest value
    float sum[1] = {0.0f};
    for (int s = 0; s < steps; ++s) {
        fetch(s);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float v[8];
            widen<BF16>(p[k], v);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[0] = fmaf(v[j], a.inv_d, sum[0]);
        }
    }
    group_sum<GROUP>(sum, part);
    const float mean = sum[0], half_mean = -0.5f * mean;
    // half of the centred value: a difference of two values of bf16's range may pass fp32's
    auto squares = [&](float scale) {
        float q[1] = {0.0f};
        for (int s = 0; s < steps; ++s) {
            if (!HELD) fetch(s);
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float v[8];
                widen<BF16>(p[k], v);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float d = fmaf(v[j], 0.5f, half_mean) * scale;
                    if (column<VEC, GROUP>(s * VPT + k, j, self) < a.D) q[0] = fmaf(d, d, q[0]);
                }
            }
        }
        group_sum<GROUP>(q, part);
        return q[0];
    };
    const float q = squares(1.0f) * a.inv_d;
    float rstd = __frsqrt_rn(fmaf(4.0f, q, a.eps));
    // squares of values above 2^63 leave fp32's range: taken again with the values scaled down
    const int over = !(q < 2e37f);
    const bool again = GROUP <= 32 ? __any_sync(0xffffffffu, over) : __syncthreads_or(over);
    if (BF16 && again) {
        const float small = squares(1.262177448353619e-29f) * a.inv_d; // 2^-96; eps does not count beside them
        if (over) rstd = __frsqrt_rn(4.0f * small) * 1.262177448353619e-29f;
    }
    if (!live) return;
    if (self == 0) {
        if (a.mean) a.mean[t] = mean;
        if (a.rstd) a.rstd[t] = rstd;
    }
    uint16_t* y = static_cast<uint16_t*>(a.y) + row * a.ldy;
    const uint16_t* w = static_cast<const uint16_t*>(a.w);
    const uint16_t* b = static_cast<const uint16_t*>(a.b);
    const float twice = 2.0f * rstd;
    for (int s = 0; s < steps; ++s) {
        if (!HELD) fetch(s);
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float v[8], g[8], c[8];
            widen<BF16>(p[k], v);
            if (w) widen<BF16>(load_row<VEC, GROUP>(w, s * VPT + k, self, a.D), g);
            if (b) widen<BF16>(load_row<VEC, GROUP>(b, s * VPT + k, self, a.D), c);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = fmaf(v[j], 0.5f, half_mean) * twice;
                if (w) v[j] *= g[j];
                if (b) v[j] += c[j];
            }
            store_row<VEC, GROUP, BF16>(y, s * VPT + k, self, a.D, v);
        }
    }
}

// The gradient: a CTA of kGradThreads on every SM, as many groups as fit in it,
// a row per group at a time.  VEC: the rows to come are copied to shared
// memory ahead, kAhead of them, each thread its own vectors, so that it waits
// for nobody's copies but its own; else the row is read where it is used.
// A group joins its two sums of a row by one barrier of its own.  16384 rows of
// 2048 bf16 elements with the residual (269 MB): NORM_GRAD_TIME.
constexpr int kGradThreads = 512;
template <int VPT> constexpr int kNormAhead = VPT == 1 ? 6 : 4;
template <int GROUP, int VPT, int VEC>
constexpr int kNormSmem = (VEC ? kNormAhead<VPT> * 3 * kGradThreads * VPT * 16 : 0) > 2 * kGradThreads * VPT * 8 * 4
                              ? kNormAhead<VPT> * 3 * kGradThreads * VPT * 16
                              : 2 * kGradThreads * VPT * 8 * 4;

template <int GROUP> __device__ __forceinline__ void group_barrier(int group)
{
    if constexpr (GROUP == 32) __syncwarp();
    else if constexpr (GROUP == kGradThreads) __syncthreads();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(GROUP) : "memory");
}

__device__ __forceinline__ void copy16(void* to, const void* from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

template <int BF16, int VEC, int GROUP, int VPT>
__global__ void __launch_bounds__(kGradThreads, 1) zero_layernorm_grad_kernel(const __grid_constant__ NormBackArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    constexpr int kGroups = kGradThreads / GROUP, kWarps = GROUP / 32, S = kNormAhead<VPT>;
    __shared__ float part[2][kGradThreads / 32][2];
    const int self = threadIdx.x % GROUP, in_cta = threadIdx.x / GROUP;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* res = static_cast<const uint16_t*>(a.res);
    uint16_t* dx = static_cast<uint16_t*>(a.dx);
    float dw[VPT][8], db[VPT][8];
    Packed w[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        if (a.w) w[k] = load_row<VEC, GROUP>(static_cast<const uint16_t*>(a.w), k, self, a.D);
        else w[k].u[0] = w[k].u[1] = w[k].u[2] = w[k].u[3] = BF16 ? 0x3f803f80u : 0x3c003c00u; // ones
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[k][j] = db[k][j] = 0.0f;
    }
    // this thread's place in slot s: three streams of VPT vectors
    auto slot = [&](int s, int stream, int k) {
        return reinterpret_cast<uint4*>(raw) + ((s * 3 + stream) * VPT + k) * kGradThreads + threadIdx.x;
    };
    auto copy_row = [&](int s, long long r) {
        if (r < a.T) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = column<1, GROUP>(k, 0, self);
                if (c >= a.D) continue;
                copy16(slot(s, 0, k), x + r * a.ldx + c);
                copy16(slot(s, 1, k), dy + r * a.lddy + c);
                if (res) copy16(slot(s, 2, k), res + r * a.ldr + c);
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    auto held = [&](int s, int stream, int k) {
        const uint4 v = *slot(s, stream, k);
        Packed p;
        p.u[0] = v.x, p.u[1] = v.y, p.u[2] = v.z, p.u[3] = v.w;
        return p;
    };
    const long long first = static_cast<long long>(blockIdx.x) * kGroups + in_cta, step = static_cast<long long>(gridDim.x) * kGroups;
    float mean_next = 0.0f, rstd_next = 0.0f;
    if (first < a.T) mean_next = a.mean[first], rstd_next = a.rstd[first];
    if constexpr (VEC) {
        // columns past the last are never copied: zeros
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int k = 0; k < VPT; ++k)
                if (column<1, GROUP>(k, 0, self) >= a.D)
                    for (int i = 0; i < 3; ++i) *slot(s, i, k) = make_uint4(0, 0, 0, 0);
        for (int s = 0; s < S - 1; ++s) copy_row(s, first + s * step);
    }
    int s = 0, turn = 0;
    for (long long r = first; r < a.T; r += step) {
        const float mean = -0.5f * mean_next, rstd = 2.0f * rstd_next;
        if (r + step < a.T) mean_next = a.mean[r + step], rstd_next = a.rstd[r + step];
        Packed px[VPT], pd[VPT], pr[VPT];
        if constexpr (VEC) {
            copy_row(s == 0 ? S - 1 : s - 1, r + (S - 1) * step); // into the slot that the last row has left
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
#pragma unroll
            for (int k = 0; k < VPT; ++k) px[k] = held(s, 0, k), pd[k] = held(s, 1, k);
        } else {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                px[k] = load_row<0, GROUP>(x + r * a.ldx, k, self, a.D);
                pd[k] = load_row<0, GROUP>(dy + r * a.lddy, k, self, a.D);
                if (res) pr[k] = load_row<0, GROUP>(res + r * a.ldr, k, self, a.D);
            }
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            float vx[8], vd[8], vw[8];
            widen<BF16>(px[k], vx);
            widen<BF16>(pd[k], vd);
            widen<BF16>(w[k], vw);
            // vectors past the last have dy 0: their sums go nowhere, so long as their h is finite
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float h = fmaf(vx[j], 0.5f, mean) * rstd;
                if (column<VEC, GROUP>(k, j, self) >= a.D) h = 0.0f;
                const float g = vd[j] * vw[j];
                dw[k][j] = fmaf(vd[j], h, dw[k][j]);
                db[k][j] += vd[j];
                sum[0] += g;
                sum[1] = fmaf(g, h, sum[1]);
            }
        }
        if (dx) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
                sum[1] += __shfl_xor_sync(0xffffffffu, sum[1], o);
            }
            if constexpr (GROUP > 32) { // two buffers in turn: a thread passes the next barrier only when all have read this one
                if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x / 32][0] = sum[0], part[turn][threadIdx.x / 32][1] = sum[1];
                group_barrier<GROUP>(in_cta);
                sum[0] = sum[1] = 0.0f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) {
                    sum[0] += part[turn][in_cta * kWarps + i][0];
                    sum[1] += part[turn][in_cta * kWarps + i][1];
                }
                turn ^= 1;
            }
            const float c0 = sum[0] * a.inv_d, c1 = sum[1] * a.inv_d, half = 0.5f * rstd;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float vx[8], vd[8], vw[8], o[8];
                widen<BF16>(px[k], vx);
                widen<BF16>(pd[k], vd);
                widen<BF16>(w[k], vw);
                if (res) {
                    if constexpr (VEC) pr[k] = held(s, 2, k);
                    widen<BF16>(pr[k], o);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float h = fmaf(vx[j], 0.5f, mean) * rstd;
                    const float d = half * (vd[j] * vw[j] - c0 - h * c1);
                    o[j] = res ? o[j] + d : d;
                }
                store_row<VEC, GROUP, BF16>(dx + r * a.lddx, k, self, a.D, o);
            }
        }
        if (++s == S) s = 0;
    }
    if (!a.sums) return;
    // the groups' sums, joined in the groups' order
    if constexpr (VEC) asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* all = reinterpret_cast<float*>(raw); // [kGroups][2][8 GROUP VPT]
    constexpr int kWidth = 8 * GROUP * VPT;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = column<VEC, GROUP>(k, j, self);
            all[(in_cta * 2) * kWidth + c] = dw[k][j];
            all[(in_cta * 2 + 1) * kWidth + c] = db[k][j];
        }
    }
    __syncthreads();
    float* to = a.sums + static_cast<long long>(blockIdx.x) * 2 * a.D;
    for (int i = threadIdx.x; i < 2 * kWidth; i += kGradThreads) {
        const int which = i / kWidth, c = i - which * kWidth;
        if (c >= a.D) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) v += all[(k * 2 + which) * kWidth + c];
        to[which * static_cast<long long>(a.D) + c] = v;
    }
}

// Rows of more than 8192 elements: dx with a CTA per row that reads it twice
// (the second time from L2), the sums of dw and db by stripes of columns.
template <int BF16, int VEC>
__global__ void __launch_bounds__(1024) zero_layernorm_wide_grad_kernel(const __grid_constant__ NormBackArgs a)
{
    constexpr int GROUP = 1024;
    __shared__ float part[GROUP / 32 * 2];
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
    const int steps = (a.D + GROUP * 8 - 1) / (GROUP * 8);
    float sum[2] = {0.0f, 0.0f};
    for (int k = 0; k < steps; ++k) {
        float vx[8], vd[8], vw[8];
        widen<BF16>(load_row<VEC, GROUP>(x, k, self, a.D), vx);
        widen<BF16>(load_row<VEC, GROUP>(dy, k, self, a.D), vd);
        if (w) widen<BF16>(load_row<VEC, GROUP>(w, k, self, a.D), vw);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (column<VEC, GROUP>(k, j, self) < a.D) {
                const float g = w ? vd[j] * vw[j] : vd[j];
                sum[0] += g;
                sum[1] = fmaf(g, fmaf(vx[j], 0.5f, mean) * rstd, sum[1]);
            }
        }
    }
    group_sum<GROUP>(sum, part);
    const float c0 = sum[0] * a.inv_d, c1 = sum[1] * a.inv_d, s = 0.5f * rstd;
    for (int k = 0; k < steps; ++k) {
        float vx[8], vd[8], vw[8], o[8];
        widen<BF16>(load_row<VEC, GROUP>(x, k, self, a.D), vx);
        widen<BF16>(load_row<VEC, GROUP>(dy, k, self, a.D), vd);
        if (w) widen<BF16>(load_row<VEC, GROUP>(w, k, self, a.D), vw);
        if (a.res) widen<BF16>(load_row<VEC, GROUP>(res, k, self, a.D), o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float g = w ? vd[j] * vw[j] : vd[j], h = fmaf(vx[j], 0.5f, mean) * rstd;
            const float d = s * (g - c0 - h * c1);
            o[j] = a.res ? o[j] + d : d;
        }
        store_row<VEC, GROUP, BF16>(dx, k, self, a.D, o);
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
        widen<BF16>(load_row<VEC, 32>(x + r * a.ldx, 0, lane, cols), vx);
        widen<BF16>(load_row<VEC, 32>(dy + r * a.lddy, 0, lane, cols), vd);
        const float mean = -0.5f * a.mean[r], rstd = 2.0f * a.rstd[r];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            dw[j] = fmaf(vd[j], fmaf(vx[j], 0.5f, mean) * rstd, dw[j]);
            db[j] += vd[j];
        }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        part[0][line][column<VEC, 32>(0, j, lane)] = dw[j];
        part[1][line][column<VEC, 32>(0, j, lane)] = db[j];
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
    int group;           // threads that share a row
};

// The narrowest group that holds a row: fewer threads have less to join; a
// warp's row needs no barrier.
template <int BF16, int VEC> NormPick pick_norm(int64_t D)
{
    if (D <= 256) return {zero_layernorm_kernel<BF16, VEC, 32, 1, 1>, 32};
    if (D <= 512) return {zero_layernorm_kernel<BF16, VEC, 32, 2, 1>, 32};
    if (D <= 1024) return {zero_layernorm_kernel<BF16, VEC, 32, 4, 1>, 32};
    if (D <= 2048) return {zero_layernorm_kernel<BF16, VEC, 256, 1, 1>, 256};
    if (D <= 4096) return {zero_layernorm_kernel<BF16, VEC, 256, 2, 1>, 256};
    if (D <= 8192) return {zero_layernorm_kernel<BF16, VEC, 256, 4, 1>, 256};
    if (D <= 16384) return {zero_layernorm_kernel<BF16, VEC, 1024, 2, 1>, 1024};
    return {zero_layernorm_kernel<BF16, VEC, 1024, 2, 0>, 1024};
}

constexpr int64_t kNormWide = 8192; // rows above it take the wide kernels

struct NormBackPick {
    NormBackKernel fn;
    int group, smem;     // threads that share a row, bytes of shared memory
};

template <int BF16, int VEC, int GROUP, int VPT> NormBackPick back_pick()
{
    return {zero_layernorm_grad_kernel<BF16, VEC, GROUP, VPT>, GROUP, kNormSmem<GROUP, VPT, VEC>};
}

template <int BF16, int VEC> NormBackPick pick_back(int64_t D)
{
    if (D <= 256) return back_pick<BF16, VEC, 32, 1>();
    if (D <= 512) return back_pick<BF16, VEC, 64, 1>();
    if (D <= 1024) return back_pick<BF16, VEC, 128, 1>();
    if (D <= 2048) return back_pick<BF16, VEC, 128, 2>();
    if (D <= 4096) return back_pick<BF16, VEC, 256, 2>();
    return back_pick<BF16, VEC, 512, 2>();
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
    NormPick k;
    if (type == ZERO_TYPE_BF16) k = vec ? pick_norm<1, 1>(D) : pick_norm<1, 0>(D);
    else k = vec ? pick_norm<0, 1>(D) : pick_norm<0, 0>(D);
    NormArgs a{};
    a.x = x, a.w = weight, a.b = bias, a.y = y, a.mean = mean, a.rstd = rstd, a.ldx = ldx, a.ldy = ldy, a.T = T;
    a.D = static_cast<int>(D), a.eps = eps, a.inv_d = 1.0f / static_cast<float>(D);
    const int threads = std::max(k.group, kNormThreads), rows = threads / k.group;
    return launch_after(k.fn, a, (T + rows - 1) / rows, threads, 0, 1, static_cast<cudaStream_t>(cuda_stream));
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
        if (dx && (rc = launch_after(rows, a, T, 1024, 0, 1, st))) return rc;
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
