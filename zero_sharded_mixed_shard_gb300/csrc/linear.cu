// The linear layer y = act(x W^T + b) + r and its gradients, on the 5th
// generation tensor cores of sm_103a.
//
// Three products share one kernel body, D[m, n] = sum_k A[m, k] B[n, k] with
// 16-bit operands and fp32 accumulators in tensor memory:
//   forward   y  = x  W^T   m = token, n = feature,  k = input
//   dx        dx = dz W     m = token, n = input,    k = feature
//   dW        dW = dz^T x   m = feature, n = input,  k = token
// An operand whose contraction index is not the contiguous one (W in dx, both
// in dW) is loaded as it lies and read by the tensor core in its "MN-major"
// form: nothing is transposed in memory.
//
// Two kernels.  zero_gemm_pair_kernel (many tiles): persistent pairs of CTAs
// that share one product of 256 rows (each holds half of the rows and half of
// the columns' operand), one TMA warp, one MMA warp, eight epilogue
// warps, accumulators doubled in tensor memory so that a tile's epilogue runs
// under the next tile's products.  zero_gemm_split_kernel (few tiles): the
// contraction is cut over the CTAs of a cluster, whose partial tiles are added
// through distributed shared memory in a fixed order; with few tokens the
// operands change sides (m = feature), so that a tile holds 128 rows of the
// weights and no more columns than tokens.  The backward pass gives both of
// its products to one launch where they take the same kernel.
//
// Every wait is bounded: one that runs out counts itself
// (zero_train_timeouts), the CTA lets its copies and products in flight end,
// frees its tensor memory and returns.
#include <cuda.h> // driver types only: the tensor-map encoder is found through the runtime
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>
#include <utility>

#include "zero_train.h"

// Defined in step.cu (not exported): keeps zero_last_cuda_error current.
__attribute__((visibility("hidden"))) int zero_record_cuda_error(int err);
// Defined in adamw.cu (not exported): the step's part of zero_train_timeouts.
__attribute__((visibility("hidden"))) int zero_adamw_wait_timeouts(unsigned int* count, int reset);

namespace {

constexpr int kGemmThreads = 384; // warp 0 TMA, warp 1 MMA, warp 2 tensor memory, warp 3 bias sums, warps 4..11 epilogue
constexpr int kEpilogueWarps = 8;
constexpr int kBM = 128;          // rows of a tile: the lanes of tensor memory
constexpr int kBK = 64;           // contraction per stage: 128 bytes, one swizzle row
constexpr int kATile = kBM * kBK * 2;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_linear_timeouts;

// Where and how a tile's results go.  swap: the tile's rows are the output's
// columns.
struct Out {
    void* y;
    void* z;             // pre-activation, may be null
    const void* bias;    // may be null
    const void* res;     // may be null
    long long ldy, ldz, ldr;
    int act, bf16, swap;
    int vec;             // 16-byte accesses allowed on y, z, res and bias
    int wide_y, wide_z, wide_r; // elements of the widest access on each: 8, 2 or 1
};

struct Problem {
    CUtensorMap a, b;
    CUtensorMap y, z;    // pairs, where o.vec: the outputs
    Out o;
    int a_mn, b_mn;      // 0: the operand's contiguous index is k; 1: it is m (n); 2: that, in whole blocks of 64
    int m, n;            // extents on the A and the B side
    int tiles_m, tiles_n;
    int kblocks;
    int cut;             // split kernel: a cluster shares each tile's contraction, else every CTA has a tile of its own
    unsigned int idesc;
};

// One launch: the tiles of one or two products, and the bias gradient's last
// sum (columns of `sums` over its chunks), which a spare warp takes along.
struct GemmArgs {
    Problem p[2];
    int tiles0, tiles;   // of the first product, of both (split kernel: its clusters)
    const float* sums;
    void* db;
    int chunks, n_db, bf16;
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ unsigned long long global_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect(uint64_t* bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes)
                 : "memory");
}

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
// or another role of the CTA has given up.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    const unsigned long long t0 = global_ns();
    for (int round = 0; round < (1 << 22); ++round) {
        for (int k = 0; k < 64; ++k)
            if (mbar_try(bar, parity)) return true;
        if (*abort) return false;
        if (global_ns() - t0 > kWaitLimitNs) break;
    }
    if (atomicExch(const_cast<int*>(abort), 1) == 0) atomicAdd(&g_linear_timeouts, 1u);
    return false;
}

// The same for copies and products in flight after a role has given up.
__device__ __noinline__ void wait_landed(uint64_t* bar, uint32_t parity)
{
    const unsigned long long t0 = global_ns();
    for (int round = 0; round < (1 << 22); ++round) {
        for (int k = 0; k < 64; ++k)
            if (mbar_try(bar, parity)) return;
        if (global_ns() - t0 > kWaitLimitNs) return;
    }
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    return mbar_try(bar, parity) || wait_slow(bar, parity, abort);
}

__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t* out, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(out)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}

__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

// The forms for a pair of CTAs: the barrier may be the other CTA's, the
// product reads both CTAs' operands, its end is told to both.
__device__ __forceinline__ uint32_t peer_addr(uint32_t local, uint32_t rank)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
    return at;
}

__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(bar)
                 : "memory");
}

// The same from a map of three dimensions: 64 contiguous elements, the
// contraction index, blocks of 64 (an MN-major operand in one instruction).
__device__ __forceinline__ void tma_load_pair3(void* dst, const CUtensorMap* map, int k, int block, uint32_t bar)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(0), "r"(k), "r"(block), "r"(bar)
                 : "memory");
}

__device__ __forceinline__ void tma_load3(void* dst, const CUtensorMap* map, int k, int block, uint64_t* bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
                 "l"(map), "r"(0), "r"(k), "r"(block), "r"(smem_addr(bar))
                 : "memory");
}

// 32 rows x 64 columns of shared memory (128-byte swizzle) to an output; what
// lies past its extents is not written.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, int x, int y, const void* src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y),
                 "r"(smem_addr(src))
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
                 : "memory");
}

__device__ __forceinline__ void mma_commit_pair(uint64_t* bar)
{
    const uint16_t both = 3;
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                     smem_addr(bar)),
                 "h"(both)
                 : "memory");
}

__device__ __forceinline__ void mbar_arrive_at(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* out, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(out)),
                 "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void tmem_free_pair(uint32_t at, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}

// Programmatic launch: everything before the wait touches only this CTA's own
// memory and runs under the preceding kernel's end; the wait returns when that
// kernel is complete and its writes are visible.
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// One lane of a converged warp.  The copy and product instructions take
// uniform registers: issued under this predicate the compiler knows that one
// thread runs them, under `lane == 0` it does not and each of them costs
// several hundred cycles (x [16384, 8192] W^T [2048], single launches: 386
// against 314 us).
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "elect.sync _|q, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void let_successor_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
                 : "memory");
}

// Arrives on `bar` when every product issued so far is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_load(uint32_t at, float (&v)[32])
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
}

__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ float4 peer_load4(uint32_t local, uint32_t rank)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(local, rank))
                 : "memory");
    return v;
}

__device__ __forceinline__ float peer_load(uint32_t local, uint32_t rank)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_addr(local, rank)) : "memory");
    return v;
}

// Shared-memory descriptor of a tile that TMA wrote with the 128-byte
// swizzle.  K-major: rows of 64 contraction elements (128 bytes), groups of 8
// rows 1024 bytes apart.  MN-major: blocks of 64 m (n) x 64 k, each k a row of
// 128 bytes, 8 of them 1024 bytes apart, the next 64 m (n) 8192 bytes on.
__device__ __forceinline__ uint64_t tile_desc(const void* p, int mn)
{
    uint64_t d = static_cast<uint64_t>((smem_addr(p) & 0x3ffff) >> 4);
    d |= static_cast<uint64_t>(mn ? 8192 >> 4 : 1) << 16;
    d |= static_cast<uint64_t>(1024 >> 4) << 32;
    d |= 1ull << 46; // descriptor version of this architecture
    d |= 2ull << 61; // 128-byte swizzle
    return d;
}

// ---------------------------------------------------------------------------
// Epilogue arithmetic
// ---------------------------------------------------------------------------

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

// GELU in tanh's form is z s(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3), and
// SiLU z s(z), with s the logistic function 1 / (1 + 2^(-x log2 e)).
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGelu = 1.5957691216057308f;
constexpr float kGelu3 = kGelu * 0.044715f;

template <int ACT> __device__ __forceinline__ float logistic(float z)
{
    const float x = ACT == ZERO_ACT_GELU ? z * fmaf(z * z, -kLog2e * kGelu3, -kLog2e * kGelu) : z * -kLog2e;
    return fast_rcp(1.0f + fast_exp2(x));
}

template <int ACT> __device__ __forceinline__ float activate(float z)
{
    if constexpr (ACT == ZERO_ACT_RELU) return z < 0.0f ? 0.0f : z; // NaN stays NaN
    else if constexpr (ACT == ZERO_ACT_NONE) return z;
    else return z * logistic<ACT>(z);
}

// The activation's derivative at z: s + z s (1 - s) u'(z).
template <int ACT> __device__ __forceinline__ float slope(float z)
{
    if constexpr (ACT == ZERO_ACT_NONE) return 1.0f;
    else {
        const float p = logistic<ACT>(z), q = fmaf(-p, p, p);
        const float d = fmaf(q, ACT == ZERO_ACT_GELU ? z * fmaf(z * z, 3.0f * kGelu3, kGelu) : z, p);
        return q == 0.0f ? p : d; // far out, where z's powers may be infinite
    }
}

// dz from dy.  ReLU's is a choice, not a product: what dy holds where z is not
// above 0, an infinity or NaN too, does not pass.
template <int ACT> __device__ __forceinline__ float through(float dy, float z)
{
    if constexpr (ACT == ZERO_ACT_RELU) return z > 0.0f ? dy : 0.0f;
    else return dy * slope<ACT>(z);
}

// N values at once: the choice of the activation stands outside the loop.
template <int N> __device__ __forceinline__ void activate_all(float (&v)[N], int act)
{
    if (act == ZERO_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = activate<ZERO_ACT_RELU>(v[j]);
    } else if (act == ZERO_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = activate<ZERO_ACT_GELU>(v[j]);
    } else if (act == ZERO_ACT_SILU) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = activate<ZERO_ACT_SILU>(v[j]);
    }
}

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

// The result in v (one or eight consecutive elements of an output row; res:
// their residual, loaded ahead).
__device__ __forceinline__ void emit(const Out& o, long long row, int col, float v, uint16_t res)
{
    if (o.bias) v += load16(o.bias, col, o.bf16);
    if (o.z) store16(o.z, row * o.ldz + col, v, o.bf16);
    float w[1] = {v};
    activate_all(w, o.act);
    if (o.res) w[0] += load16(&res, 0, o.bf16);
    store16(o.y, row * o.ldy + col, w[0], o.bf16);
}

__device__ __forceinline__ void emit8(const Out& o, long long row, int col, float (&v)[8], const uint4& res)
{
    if (o.bias) add8(v, __ldg(reinterpret_cast<const uint4*>(at16(o.bias, 0, 0, col))), o.bf16);
    if (o.z) *reinterpret_cast<uint4*>(at16(o.z, o.ldz, row, col)) = pack8(v, o.bf16);
    activate_all(v, o.act);
    if (o.res) add8(v, res, o.bf16);
    *reinterpret_cast<uint4*>(at16(o.y, o.ldy, row, col)) = pack8(v, o.bf16);
}

// A warp's 32 x 32 piece of an output, 16 bits each, in 2 KB of shared
// memory: row r's 16-byte quarter q at 4 r + (q ^ (r / 2 & 3)), so that lanes
// that hold a row each and lanes that run along rows are both free of bank
// conflicts.
__device__ __forceinline__ int piece_at(int r, int q) { return 4 * r + (q ^ ((r >> 1) & 3)); }

// `rows` x `cols` of the piece to or from memory, lanes along the rows; wide:
// elements of an access.  Rows off 16 bytes are the slow case (1009 x 1001 ->
// 1543 with residual and z: two bytes at a time 16.0 us, four 15 us; on 16
// bytes, without copies of the operands, 9 us).
__device__ __forceinline__ void piece_out(const uint4* piece, uint16_t* to, long long ld, int rows, int cols, int wide, int lane)
{
    if (cols == 32 && wide == 2) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(piece);
        const int r0 = lane >> 4, e = lane & 15;
#pragma unroll 8
        for (int r = r0; r < rows; r += 2)
            *reinterpret_cast<uint32_t*>(to + r * ld + 2 * e) = p[piece_at(r, e >> 2) * 4 + (e & 3)];
        return;
    }
    if (cols == 32 && wide == 8) {
        const int r0 = lane >> 2, q = lane & 3;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (r0 + 8 * k < rows) *reinterpret_cast<uint4*>(to + (r0 + 8 * k) * ld + q * 8) = piece[piece_at(r0 + 8 * k, q)];
    } else if (lane < cols) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(piece);
#pragma unroll 8
        for (int r = 0; r < rows; ++r) to[r * ld + lane] = p[piece_at(r, lane >> 3) * 8 + (lane & 7)];
    }
}

__device__ __forceinline__ void piece_in(uint4* piece, const uint16_t* from, long long ld, int rows, int cols, int wide, int lane)
{
    if (cols == 32 && wide > 1) {
        uint32_t* p = reinterpret_cast<uint32_t*>(piece);
        const int r0 = lane >> 4, e = lane & 15;
#pragma unroll 8
        for (int r = r0; r < rows; r += 2)
            p[piece_at(r, e >> 2) * 4 + (e & 3)] = *reinterpret_cast<const uint32_t*>(from + r * ld + 2 * e);
        return;
    }
    if (lane >= cols) return;
    uint16_t* p = reinterpret_cast<uint16_t*>(piece);
#pragma unroll 8
    for (int r = 0; r < rows; ++r) p[piece_at(r, lane >> 3) * 8 + (lane & 7)] = from[r * ld + lane];
}

// Row `lane` of the piece from this lane's 32 values.
__device__ __forceinline__ void piece_row(uint4* piece, const float (&v)[32], int bf16, int lane)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) piece[piece_at(lane, q)] = pack8(v + 8 * q, bf16);
}

// The 32 x 32 results of a warp, lane l holding row row0 + l: bias,
// pre-activation, activation, residual, and the stores.  rows, cols: how many
// exist.
template <int BF16>
__device__ __forceinline__ void emit_piece_as(const Out& o, long long row0, int rows, int col0, int cols, float (&v)[32],
                                           uint4* piece, int lane)
{
    const bool vec = o.vec && cols == 32, vec_res = o.wide_r == 8 && cols == 32;
    uint4 res[4] = {};
    if (o.res && vec_res) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if ((lane >> 2) + 8 * k < rows)
                res[k] = *reinterpret_cast<const uint4*>(at16(o.res, o.ldr, row0 + (lane >> 2) + 8 * k, col0 + (lane & 3) * 8));
    }
    if (o.bias) {
        if (vec) {
            const uint4* b = reinterpret_cast<const uint4*>(at16(o.bias, 0, 0, col0));
#pragma unroll
            for (int q = 0; q < 4; ++q) add8(v + 8 * q, __ldg(b + q), BF16);
        } else {
            const float mine = lane < cols ? load16(o.bias, col0 + lane, BF16) : 0.0f;
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, mine, j);
        }
    }
    if (o.z) {
        piece_row(piece, v, BF16, lane);
        __syncwarp();
        piece_out(piece, at16(o.z, o.ldz, row0, col0), o.ldz, rows, cols, o.wide_z, lane);
        __syncwarp();
    }
    activate_all(v, o.act);
    if (o.res) {
        if (vec_res) {
#pragma unroll
            for (int k = 0; k < 4; ++k) piece[piece_at((lane >> 2) + 8 * k, lane & 3)] = res[k];
        } else {
            piece_in(piece, at16(o.res, o.ldr, row0, col0), o.ldr, rows, cols, o.wide_r, lane);
        }
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 4; ++q) add8(v + 8 * q, piece[piece_at(lane, q)], BF16);
        __syncwarp();
    }
    piece_row(piece, v, BF16, lane);
    __syncwarp();
    piece_out(piece, at16(o.y, o.ldy, row0, col0), o.ldy, rows, cols, o.wide_y, lane);
    __syncwarp();
}

__device__ __forceinline__ void emit_piece(const Out& o, long long row0, int rows, int col0, int cols, float (&v)[32],
                                           uint4* piece, int lane)
{
    if (o.bf16) emit_piece_as<1>(o, row0, rows, col0, cols, v, piece, lane);
    else emit_piece_as<0>(o, row0, rows, col0, cols, v, piece, lane);
}

// ---------------------------------------------------------------------------
// Pieces of both kernels
// ---------------------------------------------------------------------------

__device__ __forceinline__ unsigned char* aligned_smem(unsigned char* p)
{
    return p + ((1024 - (smem_addr(p) & 1023)) & 1023);
}

// Tile t of a product: columns of kGroup m-tiles, so that the CTAs that run
// together share both operands in L2.
__device__ __forceinline__ void tile_at(const Problem& g, int t, int* mt, int* nt)
{
    constexpr int kGroup = 8;
    const int per = kGroup * g.tiles_n, group = t / per, in = t - group * per;
    const int rows = min(kGroup, g.tiles_m - group * kGroup);
    *nt = in / rows;
    *mt = group * kGroup + in - *nt * rows;
}

// The bias gradient's last sum, by warp 3 of every CTA.  A column and a step
// together may pass 2^31.  One lane adds a column's chunks, in a fixed order: with
// few columns, which have up to 760 chunks, that is the longest chain of the launch
// (backward of 4096 x 256 -> 256 22.0 us, without db 10.6; 16384 tokens 30.2, 23.9).
__device__ __forceinline__ void bias_sum(const GemmArgs& args, int lane)
{
    for (long long c = blockIdx.x * 32ll + lane; c < args.n_db; c += gridDim.x * 32ll) {
        float s = 0.0f;
#pragma unroll 16
        for (int k = 0; k < args.chunks; ++k) s += args.sums[static_cast<long long>(k) * args.n_db + c];
        store16(args.db, c, s, args.bf16);
    }
}

// ---------------------------------------------------------------------------
// Many tiles: persistent pairs of CTAs
// ---------------------------------------------------------------------------

// A pair's tile is 256 x BN: CTA r of the pair loads rows [128 r, 128 r + 128)
// of A and columns [BN/2 r, BN/2 r + BN/2) of B, and its tensor memory holds
// its 128 rows of the result.  The even CTA issues the products for both.
// Bound by the tensor cores (95 % of their cycles with 8192 inputs) and, run for
// long, by the card's power.  A pair reads 128 products for each byte it loads,
// a single CTA of 128 x 256 85, and has six stages of 64 instead of four.
// Measured: x [16384, 8192] -> 2048 with residual, fp16: 321 us for one launch
// under ncu (1710 TFLOP/s), 365 to 377 us back to back at the power limit (1480
// TFLOP/s; the library's product, without bias and residual, 349 to 356 us, so
// that it is 3 to 5 % quicker there); [8192, 2048] -> 8192
// with GELU 152 us (1810 TFLOP/s).  Eight epilogue warps: with four, GELU's
// arithmetic took longer than the products it runs under (234 us).
template <int BN> constexpr int kPairStage = kATile + BN / 2 * kBK * 2;
constexpr int kPieceBytes = 32 * 32 * 2;
constexpr int kStoreBytes = 32 * 64 * 2; // a warp's staging for stores by TMA
constexpr int kEpilogueBytes = kEpilogueWarps * kStoreBytes;

// The staging is free again once the last store has read it.  The elected lane
// is the same every time, so that it waits for its own stores.
__device__ __forceinline__ void staging_free()
{
    if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
}

// This lane's row of a half (32 columns) of the staging: 16-byte chunk q at
// q ^ (row & 7), the 128-byte swizzle.
template <int BF16> __device__ __forceinline__ void stage_row(uint4* staging, int half, const float (&v)[32], int lane)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) staging[lane * 8 + ((half * 4 + q) ^ (lane & 7))] = pack8(v + 8 * q, BF16);
}

__device__ __forceinline__ void send_staging(const CUtensorMap* map, int col, int row, const uint4* staging)
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (elect_one()) tma_store(map, col, row, staging);
    __syncwarp();
}

template <int BF16> __device__ __forceinline__ void add_bias(const Out& o, int col, float (&v)[32])
{
    if (!o.bias) return;
    const uint4* b = reinterpret_cast<const uint4*>(at16(o.bias, 0, 0, col));
#pragma unroll
    for (int q = 0; q < 4; ++q) add8(v + 8 * q, __ldg(b + q), BF16);
}

// 32 rows x 64 whole columns of a tile, from tensor memory to the outputs by
// TMA stores: the lanes only compute, and memory gets full lines (16384 x 64
// -> 8192, bf16, bound by its output: 64 us, with stores by the lanes 82 us).
// The accumulators are read a second time where the pre-activation is kept;
// `release` is called when they have been read for the last time.
template <int BF16, class Release>
__device__ __forceinline__ void emit_block_as(const Problem& g, uint32_t acc, int row0, int rows, int col, uint4* staging, int lane,
                                              Release release)
{
    const Out& o = g.o;
    if (o.z) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float v[32];
            tmem_load(acc + h * 32, v);
            add_bias<BF16>(o, col + h * 32, v);
            if (h == 0) staging_free();
            stage_row<BF16>(staging, h, v, lane);
        }
        send_staging(&g.z, col, row0, staging);
    }
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        uint4 res[4] = {};
        if (o.res) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if ((lane >> 2) + 8 * k < rows)
                    res[k] = *reinterpret_cast<const uint4*>(
                        at16(o.res, o.ldr, row0 + (lane >> 2) + 8 * k, col + h * 32 + (lane & 3) * 8));
        }
        float v[32];
        tmem_load(acc + h * 32, v);
        if (h == 1) release();
        add_bias<BF16>(o, col + h * 32, v);
        activate_all(v, o.act);
        if (h == 0) staging_free();
        if (o.res) { // lanes along the rows read it, each lane needs its own row
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = (lane >> 2) + 8 * k;
                staging[r * 8 + ((h * 4 + (lane & 3)) ^ (r & 7))] = res[k];
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) add8(v + 8 * q, staging[lane * 8 + ((h * 4 + q) ^ (lane & 7))], BF16);
        }
        stage_row<BF16>(staging, h, v, lane);
    }
    send_staging(&g.y, col, row0, staging);
}

template <class Release>
__device__ __forceinline__ void emit_block(const Problem& g, uint32_t acc, int row0, int rows, int col, uint4* staging, int lane,
                                           Release release)
{
    if (g.o.bf16) emit_block_as<1>(g, acc, row0, rows, col, staging, lane, release);
    else emit_block_as<0>(g, acc, row0, rows, col, staging, lane, release);
}

template <int BN, int STAGES, int COUNT>
__global__ void __launch_bounds__(kGemmThreads, 1) zero_gemm_pair_kernel(const __grid_constant__ GemmArgs args)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = aligned_smem(raw);
    __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem;
    __shared__ int abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31; // warp: uniform
    const int rank = static_cast<int>(cluster_rank());
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&acc_full[k], 1);
            mbar_init(&acc_empty[k], 2 * kEpilogueWarps); // the epilogue warps of both CTAs
        }
        mbar_init(&drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async;" ::: "memory");
    }
    if (warp == 2) tmem_alloc_pair(&tmem, 2 * BN);
    fence_before();
    __syncthreads();
    cluster_sync(); // the barriers are set up in both CTAs
    fence_after();
    const uint32_t base = tmem;
    volatile int* abort = &abort_flag;
    let_successor_start();
    wait_for_predecessor();

    if (warp == 0 && elect_one()) {
        int it = 0;
        bool ok = true;
        for (int t = pair; ok && t < args.tiles; t += pairs) {
            const Problem& g = args.p[COUNT == 1 ? 0 : t >= args.tiles0];
            int mt, nt;
            tile_at(g, COUNT == 2 && t >= args.tiles0 ? t - args.tiles0 : t, &mt, &nt);
            const int m0 = mt * 256 + rank * kBM, n0 = nt * BN + rank * (BN / 2);
            for (int kb = 0; kb < g.kblocks; ++kb, ++it) {
                const int s = it % STAGES;
                if (!wait(&empty[s], ((it / STAGES) & 1) ^ 1, abort)) {
                    ok = false;
                    break;
                }
                // both CTAs' copies count on the even CTA's barrier
                const uint32_t bar = peer_addr(smem_addr(&full[s]), 0);
                if (rank == 0) mbar_expect(&full[s], 2 * kPairStage<BN>);
                unsigned char* sa = smem + s * kPairStage<BN>;
                unsigned char* sb = sa + kATile;
                if (g.a_mn == 2) {
                    tma_load_pair3(sa, &g.a, kb * kBK, m0 / 64, bar);
                } else if (g.a_mn) {
                    tma_load_pair(sa, &g.a, m0, kb * kBK, bar);
                    tma_load_pair(sa + 8192, &g.a, m0 + 64, kb * kBK, bar);
                } else {
                    tma_load_pair(sa, &g.a, kb * kBK, m0, bar);
                }
                if (g.b_mn == 2) {
                    tma_load_pair3(sb, &g.b, kb * kBK, n0 / 64, bar);
                } else if (g.b_mn) {
#pragma unroll
                    for (int i = 0; i < BN / 128; ++i) tma_load_pair(sb + i * 8192, &g.b, n0 + i * 64, kb * kBK, bar);
                } else {
                    tma_load_pair(sb, &g.b, kb * kBK, n0, bar);
                }
            }
        }
        // after a wait that ran out, the copies in flight land before the CTAs end
        if (!ok && rank == 0)
            for (int k = max(0, it - STAGES); k < it; ++k) wait_landed(&full[k % STAGES], (k / STAGES) & 1);
    } else if (warp == 1 && rank == 0 && elect_one()) {
        int it = 0, n = 0;
        bool ok = true;
        for (int t = pair; ok && t < args.tiles; t += pairs, ++n) {
            const Problem& g = args.p[COUNT == 1 ? 0 : t >= args.tiles0];
            const int acc = n & 1, kblocks = g.kblocks;
            const uint64_t da = g.a_mn ? 2048 >> 4 : 32 >> 4, db = g.b_mn ? 2048 >> 4 : 32 >> 4;
            const uint64_t a0 = tile_desc(smem, g.a_mn), b0 = tile_desc(smem + kATile, g.b_mn);
            const uint32_t d = base + acc * BN, idesc = g.idesc;
            ok = wait(&acc_empty[acc], ((n >> 1) & 1) ^ 1, abort);
            fence_after();
            for (int kb = 0; ok && kb < kblocks; ++kb, ++it) {
                const int s = it % STAGES;
                if (!wait(&full[s], (it / STAGES) & 1, abort)) {
                    ok = false;
                    break;
                }
                fence_after();
                const uint64_t off = static_cast<uint64_t>(s) * (kPairStage<BN> >> 4);
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k) mma_pair(d, a0 + off + k * da, b0 + off + k * db, idesc, (kb | k) != 0);
                mma_commit_pair(&empty[s]);
            }
            if (ok) mma_commit_pair(&acc_full[acc]);
        }
        if (!ok) { // products in flight end before the tensor memory goes
            mma_commit_pair(&drained);
            wait_landed(&drained, 0);
        }
    } else if (warp == 3) {
        bias_sum(args, lane);
    } else if (warp >= 4) {
        // two warps for each 32 rows, each with half of the columns
        const int q = warp & 3, c0 = ((warp - 4) >> 2) * (BN / 2);
        uint4* staging = reinterpret_cast<uint4*>(smem + STAGES * kPairStage<BN> + (warp - 4) * kStoreBytes);
        int n = 0;
        for (int t = pair; t < args.tiles; t += pairs, ++n) {
            const Problem& g = args.p[COUNT == 1 ? 0 : t >= args.tiles0];
            int mt, nt;
            tile_at(g, COUNT == 2 && t >= args.tiles0 ? t - args.tiles0 : t, &mt, &nt);
            const int acc = n & 1;
            const bool ok = wait(&acc_full[acc], (n >> 1) & 1, abort);
            if (!__all_sync(0xffffffffu, ok)) break;
            fence_after();
            const int row0 = mt * 256 + rank * kBM + q * 32;
            const int rows = min(32, g.m - row0); // that exist; may be 0 or less
            auto release = [&] {                  // this warp's part is read: the next tile but one may have it
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(peer_addr(smem_addr(&acc_empty[acc]), 0));
            };
#pragma unroll 1
            for (int c = c0; c < c0 + BN / 2; c += 64) {
                const bool last = c + 64 == c0 + BN / 2;
                const uint32_t at = base + acc * BN + c + (static_cast<uint32_t>(q * 32) << 16);
                const int col = nt * BN + c;
                if (g.o.vec && rows > 0 && col + 64 <= g.n) {
                    emit_block(g, at, row0, rows, col, staging, lane, [&] {
                        if (last) release();
                    });
                    continue;
                }
                staging_free();
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    const int cols = min(32, g.n - (col + h * 32));
                    if (rows > 0 && cols > 0) {
                        float v[32];
                        tmem_load(at + h * 32, v);
                        emit_piece(g.o, row0, rows, col + h * 32, cols, v, staging, lane);
                    }
                }
                if (last) release();
            }
        }
        // the stores have left before the CTA ends
        if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    __syncthreads();
    __syncwarp();
    cluster_sync(); // neither CTA's memory is in use by the other any more
    fence_after();
    if (warp == 2) tmem_free_pair(base, 2 * BN);
}

// ---------------------------------------------------------------------------
// Few tiles: the contraction cut over a cluster
// ---------------------------------------------------------------------------

template <int BN> constexpr int kStageBytes = kATile + BN * kBK * 2;

// A CTA's share of joining a tile.
struct Join {
    uint32_t part;       // shared-memory address of the partial tile, the same in every CTA
    int pitch, fast, slow;
    long long row0;
    int col0, self, everyone;
    uint32_t first;      // the rank of the first partial tile
};

// Sum over the cluster's partial tiles in rank order, all of a thread's reads
// in flight together.
template <int PARTS> __device__ __forceinline__ void join(const Out& o, const Join& j)
{
    const int vecs = o.vec ? j.fast / 8 : 0; // whole vectors of 8 of a row; the rest goes element by element
    if (vecs) {
        const int total = vecs * j.slow;
        constexpr int kAhead = PARTS == 1 ? 4 : PARTS == 2 ? 2 : 1;
        for (int e = j.self; e < total; e += j.everyone * kAhead) {
            float v[kAhead][8];
            int s[kAhead], f[kAhead];
            uint4 res[kAhead] = {};
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = min(e + k * j.everyone, total - 1);
                s[k] = i / vecs;
                f[k] = (i - s[k] * vecs) * 8;
                if (o.res) res[k] = *reinterpret_cast<const uint4*>(at16(o.res, o.ldr, j.row0 + s[k], j.col0 + f[k]));
#pragma unroll
                for (int h = 0; h < 8; ++h) v[k][h] = 0.0f;
            }
            auto add = [&](int p) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const uint32_t at = j.part + static_cast<uint32_t>(s[k] * j.pitch + f[k]) * 4;
                    const float4 lo = peer_load4(at, j.first + p), hi = peer_load4(at + 16, j.first + p);
                    v[k][0] += lo.x, v[k][1] += lo.y, v[k][2] += lo.z, v[k][3] += lo.w;
                    v[k][4] += hi.x, v[k][5] += hi.y, v[k][6] += hi.z, v[k][7] += hi.w;
                }
            };
#pragma unroll
            for (int p = 0; p < PARTS; ++p) add(p);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (e + k * j.everyone < total) emit8(o, j.row0 + s[k], j.col0 + f[k], v[k], res[k]);
        }
    }
    const int left = j.fast - vecs * 8;
    if (left) {
        const int total = left * j.slow;
        constexpr int kAhead = PARTS == 8 ? 4 : 8;
        for (int e = j.self; e < total; e += j.everyone * kAhead) {
            float v[kAhead];
            int s[kAhead], f[kAhead];
            uint16_t res[kAhead] = {};
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = min(e + k * j.everyone, total - 1);
                s[k] = i / left;
                f[k] = i - s[k] * left + vecs * 8;
                if (o.res) res[k] = *at16(o.res, o.ldr, j.row0 + s[k], j.col0 + f[k]);
                v[k] = 0.0f;
            }
            auto add = [&](int p) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    v[k] += peer_load(j.part + static_cast<uint32_t>(s[k] * j.pitch + f[k]) * 4, j.first + p);
            };
#pragma unroll
            for (int p = 0; p < PARTS; ++p) add(p);
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (e + k * j.everyone < total) emit(o, j.row0 + s[k], j.col0 + f[k], v[k], res[k]);
        }
    }
}

// Bound by the reads of the weights with few tokens (4 tokens, 2048 -> 8192, bf16,
// 33.6 MB, launch included: 9.2 us from HBM, 16 weights in turn, 3650 GB/s; 7.0 us
// from L2, one weight again and again), by latency in between: launch, first
// copy, a handful of stages, join and stores follow on each other (1024 x 1024
// -> 1024 7.7 us).
// PER_SM 1: one CTA on an SM, stages as deep as they go, eight epilogue warps.
// PER_SM 2: half of all that, so that one CTA's start and end run under the
// other's products and a cluster of eight needs only four SMs.
template <int BN, int PER_SM> constexpr int kSplitThreads = PER_SM == 2 ? 256 : 384;
template <int BN, int PER_SM> constexpr int kSplitStages = PER_SM == 1 ? (BN >= 128 ? 6 : 8) : BN >= 64 ? 4 : BN >= 32 ? 5 : 6;
template <int BN, int PER_SM> constexpr int kSplitSmem = kSplitStages<BN, PER_SM> * kStageBytes<BN> + 1024;

template <int BN, int PER_SM, int COUNT>
__global__ void __launch_bounds__((kSplitThreads<BN, PER_SM>), PER_SM) zero_gemm_split_kernel(const __grid_constant__ GemmArgs args)
{
    constexpr int STAGES = kSplitStages<BN, PER_SM>, kThreads = kSplitThreads<BN, PER_SM>;
    extern __shared__ unsigned char raw[];
    unsigned char* smem = aligned_smem(raw);
    __shared__ uint64_t full[STAGES], empty[STAGES], acc_full, drained;
    __shared__ uint32_t tmem;
    __shared__ int abort_flag;
    constexpr uint32_t kCols = BN < 32 ? 32 : BN;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31; // warp: uniform
    const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
    const int cluster = blockIdx.x / size;
    const bool second = COUNT == 2 && cluster >= args.tiles0;
    const Problem& g = args.p[COUNT == 1 ? 0 : second];
    const int at = cluster - (second ? args.tiles0 : 0), t = g.cut ? at : at * size + rank;
    const bool idle = t >= g.tiles_m * g.tiles_n; // the last cluster may have CTAs without a tile
    int mt, nt;
    tile_at(g, idle ? 0 : t, &mt, &nt);
    const int parts = g.cut ? size : 1; // CTAs that share the contraction
    const int kb0 = g.cut ? static_cast<int>(static_cast<long long>(g.kblocks) * rank / parts) : 0;
    const int kb1 = g.cut ? static_cast<int>(static_cast<long long>(g.kblocks) * (rank + 1) / parts) : idle ? 0 : g.kblocks;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full, 1);
        mbar_init(&drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async;" ::: "memory");
    }
    if (warp == 2) tmem_alloc(&tmem, kCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t base = tmem;
    volatile int* abort = &abort_flag;
    let_successor_start();
    wait_for_predecessor();

    if (warp == 0 && elect_one()) {
        int it = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const int s = it % STAGES;
            if (!wait(&empty[s], ((it / STAGES) & 1) ^ 1, abort)) {
                ok = false;
                break;
            }
            mbar_expect(&full[s], kStageBytes<BN>);
            unsigned char* sa = smem + s * kStageBytes<BN>;
            unsigned char* sb = sa + kATile;
            if (g.a_mn == 2) {
                tma_load3(sa, &g.a, kb * kBK, mt * (kBM / 64), &full[s]);
            } else if (g.a_mn) {
                tma_load(sa, &g.a, mt * kBM, kb * kBK, &full[s]);
                tma_load(sa + 8192, &g.a, mt * kBM + 64, kb * kBK, &full[s]);
            } else {
                tma_load(sa, &g.a, kb * kBK, mt * kBM, &full[s]);
            }
            if (BN >= 64 && g.b_mn == 2) {
                tma_load3(sb, &g.b, kb * kBK, nt * (BN / 64), &full[s]);
            } else if (BN >= 64 && g.b_mn) {
#pragma unroll
                for (int i = 0; i < BN / 64; ++i) tma_load(sb + i * 8192, &g.b, nt * BN + i * 64, kb * kBK, &full[s]);
            } else {
                tma_load(sb, &g.b, kb * kBK, nt * BN, &full[s]);
            }
        }
        if (!ok)
            for (int k = max(0, it - STAGES); k < it; ++k) wait_landed(&full[k % STAGES], (k / STAGES) & 1);
    } else if (warp == 1 && elect_one()) {
        int it = 0;
        bool ok = true;
        const uint64_t da = g.a_mn ? 2048 >> 4 : 32 >> 4, db = g.b_mn ? 2048 >> 4 : 32 >> 4;
        const uint64_t a0 = tile_desc(smem, g.a_mn), b0 = tile_desc(smem + kATile, g.b_mn);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const int s = it % STAGES;
            if (!wait(&full[s], (it / STAGES) & 1, abort)) {
                ok = false;
                break;
            }
            fence_after();
            const uint64_t off = static_cast<uint64_t>(s) * (kStageBytes<BN> >> 4);
#pragma unroll
            for (int k = 0; k < kBK / 16; ++k) mma(base, a0 + off + k * da, b0 + off + k * db, g.idesc, kb > kb0 || k > 0);
            mma_commit(&empty[s]);
        }
        if (ok) {
            if (kb1 > kb0) mma_commit(&acc_full);
        } else {
            mma_commit(&drained);
            wait_landed(&drained, 0);
        }
    } else if (warp == 3) {
        bias_sum(args, lane);
    }
    __syncwarp();
    // The stages are free once the last product is done.
    const Out& o = g.o;
    const int rows = idle ? 0 : min(kBM, g.m - mt * kBM), cols = min(BN, g.n - nt * BN);
    float* part = reinterpret_cast<float*>(smem);
    const int pitch = (o.swap ? kBM : BN) + 4; // floats; 16-byte accesses free of bank conflicts
    const bool direct = BN >= 64 && parts == 1 && !o.swap; // nothing to join: straight from tensor memory
    // with eight epilogue warps two share 32 rows, each with half of the columns
    constexpr int kSpan = kThreads == 384 && BN >= 64 ? BN / 2 : BN;
    const int c0 = ((warp - 4) >> 2) * kSpan;
    if (warp >= 4 && kb1 > kb0 && c0 < BN) {
        const int q = warp & 3;
        const bool ok = wait(&acc_full, 0, abort);
        if (__all_sync(0xffffffffu, ok)) {
            fence_after();
            const int row = q * 32 + lane;
            const uint32_t acc = base + (static_cast<uint32_t>(q * 32) << 16);
            constexpr int kStep = BN < 32 ? 16 : 32;
#pragma unroll 1
            for (int c = c0; c < c0 + kSpan; c += kStep) {
                float v[kStep];
                if constexpr (kStep == 16) tmem_load16(acc, v);
                else tmem_load(acc + c, v);
                if constexpr (BN >= 64) {
                    if (direct) {
                        if (q * 32 < rows && c < cols)
                            emit_piece(o, mt * kBM + q * 32, min(32, rows - q * 32), nt * BN + c, min(32, cols - c), v,
                                       reinterpret_cast<uint4*>(smem + (warp - 4) * kPieceBytes), lane);
                        continue;
                    }
                }
                // the partial tile, with the output's contiguous index innermost
                if (o.swap) {
#pragma unroll
                    for (int j = 0; j < kStep; ++j) part[(c + j) * pitch + row] = v[j];
                } else {
#pragma unroll
                    for (int j = 0; j < kStep; j += 4)
                        *reinterpret_cast<float4*>(part + row * pitch + c + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
            }
            fence_before();
        }
    }
    __syncwarp();
    cluster_sync();
    if (!direct) {
        // Each CTA finishes a share of the tile: the partial sums of the
        // cluster are added in rank order.
        Join j;
        j.part = smem_addr(part);
        j.pitch = pitch;
        j.fast = o.swap ? rows : cols; // extents along and across the output's rows
        j.slow = o.swap ? cols : rows;
        j.row0 = o.swap ? nt * BN : mt * kBM;
        j.col0 = o.swap ? mt * kBM : nt * BN;
        j.first = g.cut ? 0 : static_cast<uint32_t>(rank);
        j.self = (g.cut ? rank * kThreads : 0) + static_cast<int>(threadIdx.x);
        j.everyone = (g.cut ? size : 1) * kThreads;
        switch (parts) {
        case 1: join<1>(o, j); break;
        case 2: join<2>(o, j); break;
        case 4: join<4>(o, j); break;
        default: join<8>(o, j); break;
        }
    }
    cluster_sync(); // peers have read this CTA's part
    fence_after();
    if (warp == 2) tmem_free(base, kCols);
}

// ---------------------------------------------------------------------------
// dz = dy act'(z) and the sums of its columns; copies to aligned rows
// ---------------------------------------------------------------------------

constexpr int kSumCols = 256; // columns of a CTA: 32 lanes of 8

// A matrix whose rows do not start on 16 bytes, laid out so that they do (a
// tensor map needs it).
struct Copy {
    const uint16_t* src;
    uint16_t* dst;
    long long lds, ldd, rows;
    int cols, ctas;
};

// What has to be done before the products: dz and its column sums over
// chunks of rows (`stripes` x `chunks` CTAs), and up to two copies.
struct PrepArgs {
    const void* dy;
    const void* z;
    void* dz;            // null: dz is dy
    float* sums;         // null: no bias gradient
    long long lddy, ldz, lddz, T;
    int N, rows_per, vec;
    int stripes, chunks;
    Copy copy[2];        // x, w
};

// 8 elements a thread, two bytes at a time (four-byte reads where rows allow
// them were no faster: the copies' time is latency).
__device__ __forceinline__ void copy_rows(const Copy& c, int cta)
{
    const unsigned int vecs = (c.cols + 7) / 8;
    const long long total = c.rows * vecs;
    const bool narrow = total <= 0xffffffffll; // a 64-bit division costs as much as the rest
    for (long long i = cta * 256ll + threadIdx.x; i < total; i += c.ctas * 256ll) {
        const long long r = narrow ? static_cast<unsigned int>(i) / vecs : i / vecs;
        const int at = static_cast<int>(i - r * vecs) * 8;
        const uint16_t* p = c.src + r * c.lds + at;
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = at + j < c.cols ? __ldg(p + j) : 0;
        *reinterpret_cast<uint4*>(c.dst + r * c.ldd + at) =
            make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
}

// dz is rounded to 16 bits here, once: the products' operands are 16-bit ones
// (fp32 operands would halve the tensor cores' rate and double their bytes, a
// second product with what the rounding cuts off would double the products).
// With bf16 and GELU dx and dw are off by 0.0023 of their size for it, 0.0017
// with dz in fp32, where the rounding of dx and dw themselves is left.  The
// column sums take dz before it is rounded.
// Bound by HBM and, with an activation, nearly by its arithmetic: dz and its
// sums of 8192 x 8192 bf16 with GELU 64 us (403 MB, 6300 GB/s), the sums alone
// without activation 24 us (134 MB).
template <int ACT, int BF16>
__global__ void __launch_bounds__(256) zero_linear_prep_kernel(const __grid_constant__ PrepArgs a)
{
    let_successor_start();
    wait_for_predecessor();
    int cta = blockIdx.x - a.stripes * a.chunks;
    if (cta >= 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (cta >= 0 && cta < a.copy[k].ctas) copy_rows(a.copy[k], cta);
            cta -= a.copy[k].ctas;
        }
        return;
    }
    const int stripe = blockIdx.x % a.stripes, chunk = blockIdx.x / a.stripes;
    const int lane = threadIdx.x & 31, line = threadIdx.x >> 5;
    const int col = stripe * kSumCols + lane * 8;
    const long long r0 = static_cast<long long>(chunk) * a.rows_per, r1 = min(a.T, r0 + a.rows_per);
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
    const uint16_t* z = static_cast<const uint16_t*>(a.z);
    uint16_t* dz = static_cast<uint16_t*>(a.dz);
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    if (a.vec && col + 8 <= a.N) {
        // rows a thread has in flight: 8192 x 8192, sums alone: GELU 1 row (five CTAs an SM) 53 us, 2 rows 63 us, 4 rows
        // 77 us; no activation 4 rows (four CTAs an SM) 24 us, 1 row 45 us
        constexpr int kRows = ACT == ZERO_ACT_NONE ? 4 : 1;
#pragma unroll kRows
        for (long long r = r0 + line; r < r1; r += 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(dy + r * a.lddy + col);
            uint32_t g[4] = {u.x, u.y, u.z, u.w};
            uint32_t h[4] = {};
            if (ACT != ZERO_ACT_NONE) {
                const uint4 w = *reinterpret_cast<const uint4*>(z + r * a.ldz + col);
                h[0] = w.x, h[1] = w.y, h[2] = w.z, h[3] = w.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float2 d = unpack16(g[j], BF16);
                if (ACT != ZERO_ACT_NONE) {
                    const float2 p = unpack16(h[j], BF16);
                    d.x = through<ACT>(d.x, p.x);
                    d.y = through<ACT>(d.y, p.y);
                }
                sum[2 * j] += d.x;
                sum[2 * j + 1] += d.y;
                g[j] = pack16(d.x, d.y, BF16);
            }
            if (dz) *reinterpret_cast<uint4*>(dz + r * a.lddz + col) = make_uint4(g[0], g[1], g[2], g[3]);
        }
    } else {
#pragma unroll 2
        for (long long r = r0 + line; r < r1; r += 8) {
            float d[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d[j] = 0.0f;
                if (col + j < a.N) {
                    d[j] = load16(dy, r * a.lddy + col + j, BF16);
                    if (ACT != ZERO_ACT_NONE) d[j] = through<ACT>(d[j], load16(z, r * a.ldz + col + j, BF16));
                }
                sum[j] += d[j];
            }
            // rows of dz have room for whole vectors
            if (dz && col < a.N) *reinterpret_cast<uint4*>(dz + r * a.lddz + col) = pack8(d, BF16);
        }
    }
    if (!a.sums) return;
    __shared__ float part[8][kSumCols];
#pragma unroll
    for (int j = 0; j < 8; ++j) part[line][lane * 8 + j] = sum[j];
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += part[k][threadIdx.x];
    const int c = stripe * kSumCols + threadIdx.x;
    if (c < a.N) a.sums[static_cast<long long>(chunk) * a.N + c] = s;
}

// The bias gradient's last sum where no product follows to take it along.
__global__ void __launch_bounds__(32) zero_bias_grad_kernel(const __grid_constant__ GemmArgs args)
{
    wait_for_predecessor();
    bias_sum(args, threadIdx.x);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

int record(cudaError_t e) { return e == cudaSuccess ? ZERO_OK : zero_record_cuda_error(static_cast<int>(e)); }

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

int64_t up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn tensor_map_encoder()
{
    static EncodeFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) ==
                cudaSuccess &&
            found == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeFn>(f);
    });
    return fn;
}

// A matrix [rows][ld] of 16-bit elements, cols of each row in use.
struct Matrix {
    const void* p;
    int64_t ld, rows, cols;
};

// mn 0, 1: boxes of 64 elements of `extent` rows.  mn 2: boxes of `extent`
// blocks of 64 elements of 64 rows (cols is a multiple of 64).
int make_map(CUtensorMap* map, const Matrix& x, int mn, int extent)
{
    EncodeFn encode = tensor_map_encoder();
    if (!encode) return zero_record_cuda_error(static_cast<int>(cudaErrorNotSupported));
    const cuuint64_t cols = static_cast<cuuint64_t>(x.cols), rows = static_cast<cuuint64_t>(x.rows);
    const cuuint64_t dims[3] = {mn == 2 ? 64 : cols, rows, cols / 64};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(x.ld) * 2, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(mn == 2 ? 64 : extent), static_cast<cuuint32_t>(extent)};
    const cuuint32_t step[3] = {1, 1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, mn == 2 ? 3 : 2, const_cast<void*>(x.p), dims, strides, box,
                              step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? ZERO_OK : zero_record_cuda_error(static_cast<int>(cudaErrorInvalidValue));
}

int sm_count(int* out)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    return record(e);
}

using GemmKernel = void (*)(GemmArgs);
using PrepKernel = void (*)(PrepArgs);

PrepKernel pick_prep(int act, int type)
{
    const bool b = type == ZERO_TYPE_BF16;
    switch (act) {
    case ZERO_ACT_RELU: return b ? zero_linear_prep_kernel<ZERO_ACT_RELU, 1> : zero_linear_prep_kernel<ZERO_ACT_RELU, 0>;
    case ZERO_ACT_GELU: return b ? zero_linear_prep_kernel<ZERO_ACT_GELU, 1> : zero_linear_prep_kernel<ZERO_ACT_GELU, 0>;
    case ZERO_ACT_SILU: return b ? zero_linear_prep_kernel<ZERO_ACT_SILU, 1> : zero_linear_prep_kernel<ZERO_ACT_SILU, 0>;
    default: return b ? zero_linear_prep_kernel<ZERO_ACT_NONE, 1> : zero_linear_prep_kernel<ZERO_ACT_NONE, 0>;
    }
}

// Dynamic shared memory above 48 KB is allowed once per kernel and device.
int allow_smem(GemmKernel fn, int bytes)
{
    static std::mutex mu;
    static struct { int dev; GemmKernel fn; } known[64];
    static int n_known = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record(e);
    std::lock_guard<std::mutex> lock(mu);
    for (int k = 0; k < n_known; ++k)
        if (known[k].dev == dev && known[k].fn == fn) return ZERO_OK;
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return record(e);
    if (n_known < 64) known[n_known++] = {dev, fn};
    return ZERO_OK;
}

template <int BN> constexpr int kPairStages = BN >= 256 ? 6 : 8;
template <int BN> constexpr int kPairSmem = kPairStages<BN> * kPairStage<BN> + kEpilogueBytes + 1024;

// A product to be launched: D[m, n] = sum_k A[m, k] B[n, k].
struct Product {
    Matrix a, b;
    int a_mn, b_mn;
    int64_t m, n, k;
    Out o;
};

Product product(const Matrix& a, int a_mn, const Matrix& b, int b_mn, const Out& o)
{
    return {a, b, a_mn, b_mn, a_mn ? a.cols : a.rows, b_mn ? b.cols : b.rows, a_mn ? a.rows : a.cols, o};
}

bool aligned16(const void* p, int64_t ld) { return addr(p) % 16 == 0 && ld % 8 == 0; }

// Elements of the widest access that every row start allows.
int widest_access(const void* p, int64_t ld) { return aligned16(p, ld) ? 8 : addr(p) % 4 == 0 && ld % 2 == 0 ? 2 : 1; }

// Which kernel takes a launch, with what tile.
struct Variant {
    bool pair;
    int bn, parts; // columns of a tile; CTAs that share a contraction
    int per_sm;    // CTAs on an SM
};

struct BiasSum {
    const float* sums;
    void* db;
    int chunks, n;
};

template <class Kernel, class Args>
int launch_after(Kernel fn, const Args& args, int64_t ctas, int threads, int smem, int cluster, cudaStream_t stream)
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

int64_t tiles_of(const Product& p, const Variant& v)
{
    const int64_t bm = v.pair ? 256 : kBM;
    return ((p.m + bm - 1) / bm) * ((p.n + v.bn - 1) / v.bn);
}

int64_t kblocks_of(const Product& p) { return (p.k + kBK - 1) / kBK; }

// Whether a cluster of v.parts CTAs shares a tile's contraction; one with
// fewer than two blocks a CTA is left whole.
bool is_cut(const Product& p, const Variant& v) { return v.parts > 1 && kblocks_of(p) >= 2 * v.parts; }

int64_t clusters_of(const Product& p, const Variant& v)
{
    const int64_t t = tiles_of(p, v);
    return v.pair || is_cut(p, v) ? t : (t + v.parts - 1) / v.parts;
}

// The variant with the least estimated time.  The estimates (us) are
// base + rounds of CTAs x (tail + block x blocks of 64 of the contraction),
// read off measured times, among them (tokens x inputs -> features):
//   16 columns, 2 a SM   4 x 2048 -> 8192: contraction cut in 1, 2, 4: 11.5, 8.7, 8.2
//                        4 x 8192 -> 2048: in 1, 2, 4, 8: 31.3, 18.7, 12.3, 9.3
//   64 columns, 1 a SM   1024 x 1024 -> 1024: 7.6 (2 a SM 8.7, 128 columns 8.8, pairs 12.2)
//   64 columns, 2 a SM   2048 x 1024 -> 1024: 9.2 (1 a SM 15.1: its 256 CTAs take two rounds)
//   128 columns          256 x 4096 -> 4096 cut in 1, 2, 4: 21.2, 16.4, 26.1 (pairs 26.2)
//   pairs                2048 x 2048 -> 2048: 18.6 (128 columns 25.7); 8192 x 2048 -> 8192: 156
// A second CTA on the SM (CTAs above the number of SMs) costs the first no
// time with 64 columns, and about half of its speed with fewer.
Variant choose(const Product* p, int count, int sms, double* estimate)
{
    // a tile has no more columns than the widest product needs; an MN-major operand comes in blocks of 64
    int widest = 16;
    bool swapped = false;
    for (int k = 0; k < count; ++k) {
        int bn = p[k].b_mn ? 64 : 16;
        while (bn < 128 && bn < p[k].n) bn *= 2;
        widest = std::max(widest, bn);
        swapped = swapped || p[k].o.swap;
    }
    double best = 1e30;
    Variant out{true, 256, 1, 1};
    auto consider = [&](const Variant& v, double base, double tail, double block) {
        double work = 0.0, longest = 0.0, ctas = 0.0;
        for (int k = 0; k < count; ++k) {
            const int64_t blocks = kblocks_of(p[k]);
            const double one =
                block * static_cast<double>(is_cut(p[k], v) ? (blocks + v.parts - 1) / v.parts : blocks) + tail;
            const double c = static_cast<double>(clusters_of(p[k], v)) * v.parts;
            ctas += c;
            work += one * c;
            longest = std::max(longest, one);
        }
        const double rounds = std::ceil(ctas / (v.pair ? sms / 2 : v.per_sm * sms));
        // a CTA that follows another one has its own start
        const double time = base + std::max(work / ctas * rounds, longest) + (v.pair ? 0.0 : 1.6 * (rounds - 1.0));
        if (time < best) best = time, out = v;
    };
    if (!swapped) consider({true, 256, 1, 1}, 6.3, 1.5, 0.30);
    for (int parts = 1; parts <= 8; parts *= 2) {
        const double join = std::log2(parts);
        if (widest == 128) consider({false, 128, parts, 1}, 2.2, 2.0 + 2.2 * join, 0.29);
        if (widest >= 64) {
            consider({false, 64, parts, 1}, 2.0, 1.7 + 1.5 * join, 0.25);
            consider({false, 64, parts, 2}, 2.0, 1.7 + 2.4 * join, 0.34);
        }
        if (widest <= 32) {
            const bool crowded = tiles_of(p[0], {false, widest, parts, 2}) * parts > sms;
            consider({false, widest, parts, 2}, 3.5, 2.0 + 0.3 * join, !crowded ? 0.20 : widest == 16 ? 0.35 : 0.45);
        }
    }
    *estimate = best;
    return out;
}

// Whether the gradients' two products go into launches of their own: where
// they want tiles of different shapes, one launch is not always the quicker
// form (64 tokens, 2048 -> 2048: 10 us in one, 24 in two; 4 tokens, 2048 ->
// 8192: 30 in one, 27 in two).
bool apart(const Product* p, int sms)
{
    double one, first, second;
    choose(p, 2, sms, &one);
    choose(p, 1, sms, &first);
    choose(p + 1, 1, sms, &second);
    return first + second < one;
}

// One or two products in one launch, and the bias gradient's last sum.
int gemm(const Product* p, int count, int type, const BiasSum* bias, cudaStream_t stream)
{
    int sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    double estimate;
    const Variant v = choose(p, count, sms, &estimate);
    GemmArgs args{};
    int64_t tiles = 0;
    const unsigned int t = type == ZERO_TYPE_BF16 ? 1 : 0;
    for (int k = 0; k < count; ++k) {
        Problem& g = args.p[k];
        const int bm = v.pair ? 256 : kBM, b_rows = v.pair ? v.bn / 2 : v.bn;
        g.o = p[k].o;
        g.o.wide_y = widest_access(g.o.y, g.o.ldy);
        g.o.wide_z = widest_access(g.o.z, g.o.ldz);
        g.o.wide_r = widest_access(g.o.res, g.o.ldr);
        g.o.bf16 = type == ZERO_TYPE_BF16;
        g.a_mn = p[k].a_mn ? (p[k].a.cols % 64 == 0 ? 2 : 1) : 0;
        g.b_mn = p[k].b_mn ? (p[k].b.cols % 64 == 0 ? 2 : 1) : 0;
        g.m = static_cast<int>(p[k].m);
        g.n = static_cast<int>(p[k].n);
        g.tiles_m = static_cast<int>((p[k].m + bm - 1) / bm);
        g.tiles_n = static_cast<int>((p[k].n + v.bn - 1) / v.bn);
        g.kblocks = static_cast<int>(kblocks_of(p[k]));
        g.cut = is_cut(p[k], v);
        g.idesc = (1u << 4) | (t << 7) | (t << 10) | (static_cast<unsigned int>(g.a_mn != 0) << 15) |
                  (static_cast<unsigned int>(g.b_mn != 0) << 16) | (static_cast<unsigned int>(v.bn >> 3) << 17) |
                  (static_cast<unsigned int>(bm >> 4) << 24);
        if ((rc = make_map(&g.a, p[k].a, g.a_mn, g.a_mn == 2 ? kBM / 64 : g.a_mn ? 64 : kBM))) return rc;
        if ((rc = make_map(&g.b, p[k].b, g.b_mn, g.b_mn == 2 ? b_rows / 64 : g.b_mn ? 64 : b_rows))) return rc;
        if (v.pair && g.o.vec) {
            if ((rc = make_map(&g.y, Matrix{g.o.y, g.o.ldy, p[k].m, p[k].n}, 0, 32))) return rc;
            if (g.o.z && (rc = make_map(&g.z, Matrix{g.o.z, g.o.ldz, p[k].m, p[k].n}, 0, 32))) return rc;
        }
        if (tiles_of(p[k], v) > INT32_MAX - 64) return ZERO_EINVAL;
        tiles += clusters_of(p[k], v);
        if (tiles * v.parts > INT32_MAX) return ZERO_EINVAL;
        if (k == 0) args.tiles0 = static_cast<int>(tiles);
    }
    args.tiles = static_cast<int>(tiles);
    if (bias) {
        args.sums = bias->sums;
        args.db = bias->db;
        args.chunks = bias->chunks;
        args.n_db = bias->n;
        args.bf16 = type == ZERO_TYPE_BF16;
    }
    if (v.pair) {
        GemmKernel fn = count == 1 ? zero_gemm_pair_kernel<256, kPairStages<256>, 1> : zero_gemm_pair_kernel<256, kPairStages<256>, 2>;
        if ((rc = allow_smem(fn, kPairSmem<256>))) return rc;
        return launch_after(fn, args, 2 * std::min<int64_t>(tiles, sms / 2), kGemmThreads, kPairSmem<256>, 2, stream);
    }
    GemmKernel fn = nullptr;
    int smem = 0;
    int threads = 0;
    auto pick = [&](auto columns, auto per_sm) {
        constexpr int BN = decltype(columns)::value, PER = decltype(per_sm)::value;
        fn = count == 1 ? zero_gemm_split_kernel<BN, PER, 1> : zero_gemm_split_kernel<BN, PER, 2>;
        smem = kSplitSmem<BN, PER>;
        threads = kSplitThreads<BN, PER>;
    };
    using std::integral_constant;
    if (v.bn == 16) pick(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else if (v.bn == 32) pick(integral_constant<int, 32>{}, integral_constant<int, 2>{});
    else if (v.bn == 64 && v.per_sm == 2) pick(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (v.bn == 64) pick(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else pick(integral_constant<int, 128>{}, integral_constant<int, 1>{});
    if ((rc = allow_smem(fn, smem))) return rc;
    return launch_after(fn, args, tiles * v.parts, threads, smem, v.parts, stream);
}

// Whether two strided matrices share an element.  Matrices of one row pitch
// may lie beside each other in the same rows.
bool share(const void* p, int64_t ldp, int64_t rp, int64_t cp, const void* q, int64_t ldq, int64_t rq, int64_t cq)
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

// Up to this many tokens a tile's rows are features (y) or inputs (dx), its columns tokens.
constexpr int64_t kFewTokens = 128;

constexpr int64_t kMostExtent = INT32_MAX - 512;
constexpr int64_t kMostElements = int64_t{1} << 48; // of one matrix: far above any memory, so that no size overflows

bool bad_sizes(int64_t T, int64_t K, int64_t N, int32_t act, int32_t type)
{
    return T < 0 || T > kMostExtent || K < 1 || K > kMostExtent || N < 1 || N > kMostExtent ||
           std::max(T * std::max(K, N), N * K) > kMostElements || act < ZERO_ACT_NONE || act > ZERO_ACT_SILU ||
           (type != ZERO_TYPE_FP16 && type != ZERO_TYPE_BF16);
}

// Whether a matrix has a byte in the used part of the workspace.
bool in_workspace(const void* ws, int64_t used, const void* p, int64_t ld, int64_t rows, int64_t cols)
{
    if (!p || rows < 1) return false;
    const uintptr_t end = addr(p) + (static_cast<uintptr_t>(rows - 1) * ld + cols) * 2;
    return addr(p) < addr(ws) + static_cast<uintptr_t>(used) && addr(ws) < end;
}

constexpr int64_t kMostLd = int64_t{1} << 38;

bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > kMostLd; }

// Rows of a chunk of the column sums: four CTAs per SM, five (all that fit)
// where an activation's arithmetic wants the warps, and at least 8 rows.
int sum_rows(int64_t T, int64_t N, int act)
{
    const int64_t stripes = (N + kSumCols - 1) / kSumCols;
    const int64_t want = std::max<int64_t>(1, (act == ZERO_ACT_NONE ? 608 : 760) / stripes);
    return static_cast<int>(std::max<int64_t>(8, up((T + want - 1) / want, 8)));
}

int64_t sum_chunks(int64_t T, int64_t N, int act)
{
    const int64_t r = sum_rows(T, N, act);
    return std::max<int64_t>(1, (T + r - 1) / r);
}

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

int64_t matrix_bytes(int64_t rows, int64_t cols) { return rows * up(cols, 8) * 2; }

// Adds the copy of x to rows on 16 bytes to a launch of the preparing kernel.
void add_copy(PrepArgs* a, int* ctas, int slot, Matrix* x, void* to)
{
    const int64_t ld = up(x->cols, 8), vecs = x->rows * (ld / 8);
    Copy& c = a->copy[slot];
    c.src = static_cast<const uint16_t*>(x->p);
    c.dst = static_cast<uint16_t*>(to);
    c.lds = x->ld;
    c.ldd = ld;
    c.rows = x->rows;
    c.cols = static_cast<int>(x->cols);
    c.ctas = static_cast<int>(std::min<int64_t>(4864, (vecs + 255) / 256));
    *ctas += c.ctas;
    x->p = to;
    x->ld = ld;
}

} // namespace

extern "C" int zero_linear_plan(int64_t T, int64_t K, int64_t N, int32_t products, int32_t* launches, int32_t* rows,
                                int32_t* columns, int32_t* cluster, int32_t* per_sm)
{
    if (!launches || !rows || !columns || !cluster || !per_sm || products < 0 || products > 3 || T < 1 ||
        bad_sizes(T, K, N, ZERO_ACT_NONE, ZERO_TYPE_FP16))
        return ZERO_EINVAL;
    int sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    const Matrix x{nullptr, K, T, K}, w{nullptr, K, N, K}, dz{nullptr, N, T, N};
    Out o{};
    o.swap = T <= kFewTokens;
    Product p[2];
    int count = 0;
    if (products == 0) p[count++] = o.swap ? product(w, 0, x, 0, o) : product(x, 0, w, 0, o);
    if (products & 1) p[count++] = o.swap ? product(w, 1, dz, 0, o) : product(dz, 0, w, 1, o);
    o.swap = 0;
    if (products & 2) p[count++] = product(dz, 1, x, 1, o);
    *launches = count == 2 && apart(p, sms) ? 2 : 1;
    double estimate;
    const Variant v = choose(p, *launches == 2 ? 1 : count, sms, &estimate);
    *rows = v.pair ? 256 : kBM;
    *columns = v.bn;
    *cluster = v.pair ? 2 : v.parts;
    *per_sm = v.per_sm;
    return ZERO_OK;
}

extern "C" int zero_linear_workspace(int64_t T, int64_t K, int64_t N, int32_t act, int32_t backward, int32_t aligned,
                                     int64_t* bytes)
{
    if (!bytes || bad_sizes(T, K, N, act, ZERO_TYPE_FP16)) return ZERO_EINVAL;
    Carver c{nullptr};
    if (!aligned) {
        c.take(matrix_bytes(T, K));
        c.take(matrix_bytes(N, K));
    }
    if (backward) {
        if (act != ZERO_ACT_NONE || !aligned) c.take(matrix_bytes(T, N));
        c.take(sum_chunks(T, N, act) * N * 4);
    }
    *bytes = c.used;
    return ZERO_OK;
}

extern "C" int zero_linear_forward(const void* x, int64_t ldx, const void* w, int64_t ldw, const void* bias,
                                   const void* residual, int64_t ldr, void* y, int64_t ldy, void* z, int64_t ldz,
                                   int64_t T, int64_t K, int64_t N, int32_t act, int32_t type, void* workspace,
                                   int64_t workspace_bytes, void* cuda_stream)
{
    if (bad_sizes(T, K, N, act, type)) return ZERO_EINVAL;
    if (T == 0) return ZERO_OK;
    if (!x || !w || !y || bad_ld(ldx, K) || bad_ld(ldw, K) || bad_ld(ldy, N) || (z && bad_ld(ldz, N)) ||
        (residual && bad_ld(ldr, N)))
        return ZERO_EINVAL;
    for (const void* p : {x, w, bias, residual, static_cast<const void*>(y), static_cast<const void*>(z)})
        if (addr(p) % 2) return ZERO_EALIGN;
    for (int k = 0; k < 2; ++k) { // the outputs y and z
        const void* p = k ? z : y;
        const int64_t ld = k ? ldz : ldy;
        if (share(p, ld, T, N, x, ldx, T, K) || share(p, ld, T, N, w, ldw, N, K) || share(p, ld, T, N, bias, N, 1, N))
            return ZERO_EOVERLAP;
        const bool same = !k && residual == y && ldr == ldy; // in place: each element is read before it is written
        if (residual && !same && share(p, ld, T, N, residual, ldr, T, N)) return ZERO_EOVERLAP;
    }
    if (share(y, ldy, T, N, z, ldz, T, N)) return ZERO_EOVERLAP;

    Matrix mx{x, ldx, T, K}, mw{w, ldw, N, K};
    const bool fix_x = !aligned16(x, ldx), fix_w = !aligned16(w, ldw);
    Carver c{static_cast<unsigned char*>(workspace)};
    void* tx = fix_x ? c.take(matrix_bytes(T, K)) : nullptr;
    void* tw = fix_w ? c.take(matrix_bytes(N, K)) : nullptr;
    if (c.used > 0) {
        if (!workspace || workspace_bytes < c.used) return ZERO_EINVAL;
        if (addr(workspace) % 16) return ZERO_EALIGN;
        const Matrix all[] = {{x, ldx, T, K}, {w, ldw, N, K}, {bias, N, 1, N}, {residual, ldr, T, N}, {y, ldy, T, N}, {z, ldz, T, N}};
        for (const Matrix& q : all)
            if (in_workspace(workspace, c.used, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    int rc = ZERO_OK, ctas = 0;
    PrepArgs prep{};
    if (fix_x) add_copy(&prep, &ctas, 0, &mx, tx);
    if (fix_w) add_copy(&prep, &ctas, 1, &mw, tw);
    if (ctas && (rc = launch_after(pick_prep(ZERO_ACT_NONE, type), prep, ctas, 256, 0, 1, st))) return rc;
    Out o{};
    o.y = y, o.ldy = ldy, o.z = z, o.ldz = ldz, o.bias = bias, o.res = residual, o.ldr = ldr, o.act = act;
    o.vec = aligned16(y, ldy) && (!z || aligned16(z, ldz)) && (!residual || aligned16(residual, ldr)) && addr(bias) % 16 == 0;
    o.swap = T <= kFewTokens;
    const Product p = o.swap ? product(mw, 0, mx, 0, o) : product(mx, 0, mw, 0, o);
    return gemm(&p, 1, type, nullptr, st);
}

extern "C" int zero_linear_backward(const void* dy, int64_t lddy, const void* z, int64_t ldz, const void* x, int64_t ldx,
                                    const void* w, int64_t ldw, void* dx, int64_t lddx, void* dw, int64_t lddw, void* db,
                                    int64_t T, int64_t K, int64_t N, int32_t act, int32_t type, void* workspace,
                                    int64_t workspace_bytes, void* cuda_stream)
{
    if (bad_sizes(T, K, N, act, type)) return ZERO_EINVAL;
    if (!dx && !dw && !db) return ZERO_EINVAL;
    if (dw && bad_ld(lddw, K)) return ZERO_EINVAL;
    if (T > 0) {
        if (!dy || bad_ld(lddy, N) || (act != ZERO_ACT_NONE && (!z || bad_ld(ldz, N))) || (dx && (!w || bad_ld(ldw, K))) ||
            (dw && (!x || bad_ld(ldx, K))) || (dx && bad_ld(lddx, K)))
            return ZERO_EINVAL;
    }
    if (act == ZERO_ACT_NONE) z = nullptr;
    if (!dx) w = nullptr;
    if (!dw) x = nullptr;
    for (const void* p : {dy, z, x, w, static_cast<const void*>(dx), static_cast<const void*>(dw), static_cast<const void*>(db)})
        if (addr(p) % 2) return ZERO_EALIGN;
    struct { const void* p; int64_t ld, rows, cols; } out[3] = {{dx, lddx, T, K}, {dw, lddw, N, K}, {db, N, 1, N}},
        in[4] = {{dy, lddy, T, N}, {z, ldz, T, N}, {x, ldx, T, K}, {w, ldw, N, K}};
    for (int i = 0; i < 3; ++i) {
        for (const auto& q : in)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
        for (int j = i + 1; j < 3; ++j)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, out[j].p, out[j].ld, out[j].rows, out[j].cols))
                return ZERO_EOVERLAP;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (T == 0) { // sums over no tokens
        cudaError_t e = cudaSuccess;
        if (dw) e = cudaMemset2DAsync(dw, static_cast<size_t>(lddw) * 2, 0, static_cast<size_t>(K) * 2, static_cast<size_t>(N), st);
        if (db && e == cudaSuccess) e = cudaMemsetAsync(db, 0, static_cast<size_t>(N) * 2, st);
        return record(e);
    }

    const bool has_act = act != ZERO_ACT_NONE, products = dx || dw;
    const bool fix_x = dw && !aligned16(x, ldx), fix_w = dx && !aligned16(w, ldw);
    const bool make_dz = products && (has_act || !aligned16(dy, lddy));
    Carver c{static_cast<unsigned char*>(workspace)};
    void* tx = fix_x ? c.take(matrix_bytes(T, K)) : nullptr;
    void* tw = fix_w ? c.take(matrix_bytes(N, K)) : nullptr;
    void* tz = make_dz ? c.take(matrix_bytes(T, N)) : nullptr;
    const int64_t chunks = sum_chunks(T, N, act);
    float* sums = db ? static_cast<float*>(c.take(chunks * N * 4)) : nullptr;
    if (c.used > 0) {
        if (!workspace || workspace_bytes < c.used) return ZERO_EINVAL;
        if (addr(workspace) % 16) return ZERO_EALIGN;
        for (const auto& q : in)
            if (in_workspace(workspace, c.used, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
        for (const auto& q : out)
            if (in_workspace(workspace, c.used, q.p, q.ld, q.rows, q.cols)) return ZERO_EOVERLAP;
    }
    Matrix mx{x, ldx, T, K}, mw{w, ldw, N, K}, mz{dy, lddy, T, N};
    int rc = ZERO_OK, ctas = 0;
    PrepArgs prep{};
    if (make_dz || db) {
        prep.dy = dy, prep.lddy = lddy, prep.z = z, prep.ldz = ldz, prep.dz = tz, prep.lddz = up(N, 8), prep.sums = sums;
        prep.T = T, prep.N = static_cast<int>(N), prep.rows_per = sum_rows(T, N, act);
        prep.vec = aligned16(dy, lddy) && (!has_act || aligned16(z, ldz));
        prep.stripes = static_cast<int>((N + kSumCols - 1) / kSumCols);
        prep.chunks = static_cast<int>(chunks);
        if (chunks * prep.stripes > INT32_MAX - 4096) return ZERO_EINVAL;
        ctas = prep.stripes * prep.chunks;
        if (make_dz) mz = {tz, up(N, 8), T, N};
    }
    if (fix_x) add_copy(&prep, &ctas, 0, &mx, tx);
    if (fix_w) add_copy(&prep, &ctas, 1, &mw, tw);
    if (ctas && (rc = launch_after(pick_prep(act, type), prep, ctas, 256, 0, 1, st))) return rc;

    const BiasSum bias{sums, db, static_cast<int>(chunks), static_cast<int>(N)};
    if (!products) {
        GemmArgs args{};
        args.sums = sums, args.db = db, args.chunks = bias.chunks, args.n_db = bias.n, args.bf16 = type == ZERO_TYPE_BF16;
        return launch_after(zero_bias_grad_kernel, args, (N + 31) / 32, 32, 0, 1, st);
    }
    Product p[2];
    int count = 0;
    if (dx) {
        Out o{};
        o.y = dx, o.ldy = lddx, o.vec = aligned16(dx, lddx), o.swap = T <= kFewTokens;
        p[count++] = o.swap ? product(mw, 1, mz, 0, o) : product(mz, 0, mw, 1, o);
    }
    if (dw) {
        Out o{};
        o.y = dw, o.ldy = lddw, o.vec = aligned16(dw, lddw);
        p[count++] = product(mz, 1, mx, 1, o);
    }
    const BiasSum* with = db ? &bias : nullptr;
    int sms = 0;
    if ((rc = sm_count(&sms))) return rc;
    if (count == 2 && apart(p, sms)) {
        if ((rc = gemm(p, 1, type, with, st))) return rc;
        return gemm(p + 1, 1, type, nullptr, st);
    }
    if (count == 2 && kblocks_of(p[1]) > kblocks_of(p[0])) std::swap(p[0], p[1]); // the longer tiles first
    return gemm(p, count, type, with, st);
}

extern "C" int zero_train_timeouts(int64_t* count, int32_t reset)
{
    if (!count) return ZERO_EINVAL;
    unsigned int n = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&n, g_linear_timeouts, sizeof(n));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_linear_timeouts, &zero, sizeof(zero));
    }
    if (e != cudaSuccess) return record(e);
    unsigned int steps = 0;
    const int rc = zero_adamw_wait_timeouts(&steps, reset);
    if (rc) return rc;
    *count = static_cast<int64_t>(n) + steps;
    return ZERO_OK;
}
