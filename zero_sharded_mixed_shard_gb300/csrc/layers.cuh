// Shared by the layers' translation units: 16-bit conversions, programmatic
// launches, and the host's checks of strided matrices and workspaces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "zero_train.h"

// Defined in step.cu (not exported): keeps zero_last_cuda_error current.
__attribute__((visibility("hidden"))) int zero_record_cuda_error(int err);

namespace {

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Programmatic launch: everything before the wait touches only this CTA's own
// memory and runs under the preceding kernel's end; the wait returns when that
// kernel is complete and its writes are visible.
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float load16(const void* p, long long i, int bf16)
{
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store16(void* p, long long i, float v, int bf16)
{
    if (bf16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half*>(p)[i] = __float2half_rn(v);
}

__device__ __forceinline__ uint32_t pack16(float a, float b, int bf16)
{
    if (bf16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack16(uint32_t u, int bf16)
{
    if (bf16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// 2^x and 1 / x by the hardware's approximations (2 and 1 ulp).
__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fast_rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void add8(float* v, const uint4& u, int bf16)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(w[j], bf16);
        v[2 * j] += f.x;
        v[2 * j + 1] += f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float* v, int bf16)
{
    return make_uint4(pack16(v[0], v[1], bf16), pack16(v[2], v[3], bf16), pack16(v[4], v[5], bf16), pack16(v[6], v[7], bf16));
}

__device__ __forceinline__ uint16_t* at16(const void* p, long long ld, long long row, int col)
{
    return static_cast<uint16_t*>(const_cast<void*>(p)) + row * ld + col;
}

// ---------------------------------------------------------------------------
// Rows that start anywhere: reads and writes by whole 16-byte granules
// ---------------------------------------------------------------------------

// Elements before p in its 16-byte granule.
__device__ __forceinline__ int phase_of(const uint16_t* p) { return static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15) >> 1; }

// Elements e .. e + 7 of the sixteen in a and b, 0 <= e < 8.
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b, int e)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 6; ++j) w[j] = e & 4 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) w[j] = e & 2 ? w[j + 1] : w[j];
    const int half = (e & 1) * 16;
    return make_uint4(__funnelshift_r(w[0], w[1], half), __funnelshift_r(w[1], w[2], half), __funnelshift_r(w[2], w[3], half),
                      __funnelshift_r(w[3], w[4], half));
}

// The first n of eight elements, zeros behind them.
__device__ __forceinline__ uint4 first_of(const uint4& v, int n)
{
    if (n >= 8) return v;
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = n >= 2 * j + 2 ? w[j] : n == 2 * j + 1 ? w[j] & 0xffffu : 0u;
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Elements [c, c + 8) of a row of D, c above -8, zeros past its end (what lies
// before the row is anything).  Reads only granules that hold an element of
// the row.
__device__ __forceinline__ uint4 load_any(const uint16_t* row, int c, int D)
{
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    const int e = phase_of(row + c);
    const uint4* from = reinterpret_cast<const uint4*>(row + c - e);
    if (c < D && c - e > -8) a = from[0];
    if (e && c + 8 - e < D) b = from[1];
    return first_of(shifted(a, b, e), D - c);
}

// The first n (0 to 7) elements of a granule, and those from e (1 to 7) on, in
// three stores at most.
__device__ __forceinline__ void put_first(uint16_t* p, const uint4& g, int n)
{
    if (n & 4) *reinterpret_cast<uint2*>(p) = make_uint2(g.x, g.y);
    if (n & 2) *reinterpret_cast<uint32_t*>(p + (n & 4)) = n & 4 ? g.z : g.x;
    if (n & 1) p[n - 1] = static_cast<uint16_t>(n & 4 ? (n & 2 ? g.w : g.z) : (n & 2 ? g.y : g.x));
}

__device__ __forceinline__ void put_from(uint16_t* p, const uint4& g, int e)
{
    if (e <= 4) *reinterpret_cast<uint2*>(p + 4) = make_uint2(g.z, g.w);
    if (e <= 2 || e == 5 || e == 6) *reinterpret_cast<uint32_t*>(p + (e <= 2 ? 2 : 6)) = e <= 2 ? g.y : g.w;
    if (e & 1) p[e] = static_cast<uint16_t>((e & 4 ? (e & 2 ? g.w : g.z) : (e & 2 ? g.y : g.x)) >> 16);
}

// The granule whose first element is `at` (above -8) of a row of D: what
// belongs to the row.
__device__ __forceinline__ void put_granule(uint16_t* row, int at, int D, const uint4& g)
{
    uint16_t* p = row + at;
    if (at >= 0 && at + 8 <= D) {
        *reinterpret_cast<uint4*>(p) = g;
    } else if (at >= 0) {
        if (at < D) put_first(p, g, D - at);
    } else if (at + 8 <= D) {
        put_from(p, g, -at);
    } else { // a row that begins and ends in one granule
        const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (at + j >= 0 && at + j < D) p[j] = static_cast<uint16_t>(w[j >> 1] >> (j & 1) * 16);
    }
}

// Elements [c, c + 8) of a row of D from each of a run of lanes with
// neighbouring c, by whole warps; `first` and `last` mark the run's ends.  A
// granule is written whole where the run holds all of it.
__device__ __forceinline__ void store_any(uint16_t* row, int c, int D, const uint4& v, bool first, bool last)
{
    const int e = phase_of(row + c), at = c - e;
    uint4 before;
    before.x = __shfl_up_sync(0xffffffffu, v.x, 1);
    before.y = __shfl_up_sync(0xffffffffu, v.y, 1);
    before.z = __shfl_up_sync(0xffffffffu, v.z, 1);
    before.w = __shfl_up_sync(0xffffffffu, v.w, 1);
    const uint4 g = e ? shifted(before, v, 8 - e) : v; // the granule that holds element c
    uint16_t* p = row + at;
    if (at + 8 <= D && (!first || !e)) {
        *reinterpret_cast<uint4*>(p) = g;
    } else if (!first || !e) {
        if (at < D) put_first(p, g, D - at);
    } else if (at + 8 <= D) {
        put_from(p, g, e);
    } else { // a row that begins and ends in one granule
        const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
        for (int j = 1; j < 8; ++j)
            if (j >= e && at + j < D) p[j] = static_cast<uint16_t>(w[j >> 1] >> (j & 1) * 16);
    }
    if (last && e && at + 8 < D) put_first(p + 8, shifted(v, make_uint4(0, 0, 0, 0), 8 - e), min(e, D - at - 8));
}

// ---------------------------------------------------------------------------
// Two fp32 operations in one instruction
// ---------------------------------------------------------------------------

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\tfma.rn.f32x2 a, a, b, c;\n\t"
        "mov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

inline int record(cudaError_t e) { return e == cudaSuccess ? ZERO_OK : zero_record_cuda_error(static_cast<int>(e)); }

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

inline int64_t up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

inline int sm_count(int* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    return record(e);
}

inline bool aligned16(const void* p, int64_t ld) { return addr(p) % 16 == 0 && ld % 8 == 0; }

// Elements of the widest access that every row start allows.
inline int widest_access(const void* p, int64_t ld) { return aligned16(p, ld) ? 8 : addr(p) % 4 == 0 && ld % 2 == 0 ? 2 : 1; }

// Dynamic shared memory above 48 KB is allowed once per kernel and device.
inline int allow_smem(const void* fn, int bytes)
{
    static std::mutex mu;
    static struct { int dev; const void* fn; } known[128];
    static int n_known = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record(e);
    std::lock_guard<std::mutex> lock(mu);
    for (int k = 0; k < n_known; ++k)
        if (known[k].dev == dev && known[k].fn == fn) return ZERO_OK;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return record(e);
    if (n_known < 128) known[n_known++] = {dev, fn};
    return ZERO_OK;
}

// A launch whose start may overlap the preceding kernel's end.
template <class Kernel, class Args>
inline int launch_after(Kernel fn, const Args& args, int64_t ctas, int threads, int smem, int cluster, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned int>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned int>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = static_cast<unsigned int>(cluster);
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return record(cudaLaunchKernelEx(&cfg, fn, args));
}

// Whether two strided matrices share an element.  Matrices of one row pitch
// may lie beside each other in the same rows.
inline bool share(const void* p, int64_t ldp, int64_t rp, int64_t cp, const void* q, int64_t ldq, int64_t rq, int64_t cq)
{
    if (!p || !q || rp < 1 || rq < 1) return false;
    const uintptr_t pe = addr(p) + (static_cast<uintptr_t>(rp - 1) * ldp + cp) * 2;
    const uintptr_t qe = addr(q) + (static_cast<uintptr_t>(rq - 1) * ldq + cq) * 2;
    if (addr(p) >= qe || addr(q) >= pe) return false;
    if (ldp != ldq) return true;
    const uintptr_t pitch = static_cast<uintptr_t>(ldp) * 2;
    // q's first column, counted from p's within a row
    const uintptr_t d = addr(q) >= addr(p) ? (addr(q) - addr(p)) % pitch : (pitch - (addr(p) - addr(q)) % pitch) % pitch;
    return !(d >= static_cast<uintptr_t>(cp) * 2 && pitch - d >= static_cast<uintptr_t>(cq) * 2);
}

constexpr int64_t kMostExtent = INT32_MAX - 512;

constexpr int64_t kMostElements = int64_t{1} << 48; // of one matrix: far above any memory, so that no size overflows

inline bool bad_sizes(int64_t T, int64_t K, int64_t N, int32_t act, int32_t type)
{
    return T < 0 || T > kMostExtent || K < 1 || K > kMostExtent || N < 1 || N > kMostExtent ||
           std::max(T * std::max(K, N), N * K) > kMostElements || act < ZERO_ACT_NONE || act > ZERO_ACT_SILU ||
           (type != ZERO_TYPE_FP16 && type != ZERO_TYPE_BF16);
}

// Whether a matrix has a byte in the used part of the workspace.
inline bool in_workspace(const void* ws, int64_t used, const void* p, int64_t ld, int64_t rows, int64_t cols)
{
    if (!p || rows < 1) return false;
    const uintptr_t end = addr(p) + (static_cast<uintptr_t>(rows - 1) * ld + cols) * 2;
    return addr(p) < addr(ws) + static_cast<uintptr_t>(used) && addr(ws) < end;
}

constexpr int64_t kMostLd = int64_t{1} << 38;

inline bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > kMostLd; }

// A piece of the caller's workspace, on 256 bytes.
struct Carver {
    unsigned char* base;
    int64_t used = 0;
    void* take(int64_t bytes)
    {
        void* p = base ? base + used : nullptr;
        used += up(bytes, 256);
        return p;
    }
};

inline int64_t matrix_bytes(int64_t rows, int64_t cols) { return rows * up(cols, 8) * 2; }

} // namespace
