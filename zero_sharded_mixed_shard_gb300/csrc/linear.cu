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
// Two kernels.  zero_gemm_kernel (many tiles): persistent CTAs, one TMA warp,
// one MMA warp, four epilogue warps, accumulators doubled in tensor memory so
// that a tile's epilogue runs under the next tile's products.
// zero_gemm_split_kernel (few tiles): the contraction is cut over the CTAs of
// a cluster, whose partial tiles are added through distributed shared memory
// in a fixed order; with few tokens the operands change sides (m = feature),
// so that a tile holds 128 rows of the weights and no more columns than
// tokens.
//
// Every wait is bounded: one that runs out counts itself
// (zero_linear_timeouts), the CTA lets its copies and products in flight end,
// frees its tensor memory and returns.
#include <cuda.h> // driver types only: the tensor-map encoder is found through the runtime
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

constexpr int kGemmThreads = 256; // warp 0 TMA, warp 1 MMA, warp 2 tensor memory, warps 4..7 epilogue
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
    int rows, cols;      // of the output
    int act, bf16, swap;
    int vec;             // 16-byte accesses allowed on y, z, res and bias rows
};

struct GemmArgs {
    CUtensorMap a, b;
    Out o;
    int a_mn, b_mn;      // the operand's contiguous index is m (n), not k
    int m, n;            // extents on the A and the B side
    int tiles_m, tiles_n;
    int kblocks;
    unsigned int idesc;
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

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
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

__device__ __forceinline__ float peer_load(uint32_t local, uint32_t rank)
{
    uint32_t at;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
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

// 2 sqrt(2 / pi): tanh's form of GELU is z / (1 + exp(-kGelu (z + 0.044715 z^3))).
constexpr float kGelu = 1.5957691216057308f;
constexpr float kCube = 0.044715f;

__device__ __forceinline__ float activate(float z, int act)
{
    if (act == ZERO_ACT_RELU) return z > 0.0f ? z : 0.0f;
    if (act == ZERO_ACT_GELU) return __fdividef(z, 1.0f + __expf(-kGelu * (z + kCube * z * z * z)));
    if (act == ZERO_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
    return z;
}

// The activation's derivative at z.
__device__ __forceinline__ float slope(float z, int act)
{
    if (act == ZERO_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if (act == ZERO_ACT_GELU) {
        const float p = __fdividef(1.0f, 1.0f + __expf(-kGelu * (z + kCube * z * z * z)));
        return p + z * p * (1.0f - p) * kGelu * (1.0f + 3.0f * kCube * z * z);
    }
    if (act == ZERO_ACT_SILU) {
        const float p = __fdividef(1.0f, 1.0f + __expf(-z));
        return p + z * p * (1.0f - p);
    }
    return 1.0f;
}

// One output element from its accumulator.
__device__ __forceinline__ void emit(const Out& o, int row, int col, float v)
{
    if (o.bias) v += load16(o.bias, col, o.bf16);
    if (o.z) store16(o.z, row * o.ldz + col, v, o.bf16);
    v = activate(v, o.act);
    if (o.res) v += load16(o.res, row * o.ldr + col, o.bf16);
    store16(o.y, row * o.ldy + col, v, o.bf16);
}

// 32 consecutive elements of an output row, from column col on.
__device__ __forceinline__ void emit32(const Out& o, long long row, int col, float (&v)[32])
{
    if (!o.vec || col + 32 > o.cols) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (col + j < o.cols) emit(o, static_cast<int>(row), col + j, v[j]);
        return;
    }
    if (o.bias) {
        const uint4* b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(o.bias) + col);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 u = __ldg(b + q);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack16(w[j], o.bf16);
                v[q * 8 + 2 * j] += f.x;
                v[q * 8 + 2 * j + 1] += f.y;
            }
        }
    }
    auto store = [&](void* base, long long ld) {
        uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + row * ld + col);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            p[q] = make_uint4(pack16(v[q * 8], v[q * 8 + 1], o.bf16), pack16(v[q * 8 + 2], v[q * 8 + 3], o.bf16),
                              pack16(v[q * 8 + 4], v[q * 8 + 5], o.bf16), pack16(v[q * 8 + 6], v[q * 8 + 7], o.bf16));
    };
    if (o.z) store(o.z, o.ldz);
    if (o.act != ZERO_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = activate(v[j], o.act);
    }
    if (o.res) {
        const uint4* r = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(o.res) + row * o.ldr + col);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 u = r[q];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = unpack16(w[j], o.bf16);
                v[q * 8 + 2 * j] += f.x;
                v[q * 8 + 2 * j + 1] += f.y;
            }
        }
    }
    store(o.y, o.ldy);
}

// ---------------------------------------------------------------------------
// Pieces of both kernels
// ---------------------------------------------------------------------------

template <int BN> constexpr int kStageBytes = kATile + BN * kBK * 2;

template <int BN>
__device__ __forceinline__ void load_stage(const GemmArgs& g, unsigned char* stage, uint64_t* bar, int mt, int nt, int kb)
{
    mbar_expect(bar, kStageBytes<BN>);
    unsigned char* sb = stage + kATile;
    if (g.a_mn) {
#pragma unroll
        for (int i = 0; i < kBM / 64; ++i) tma_load(stage + i * 8192, &g.a, mt * kBM + i * 64, kb * kBK, bar);
    } else {
        tma_load(stage, &g.a, kb * kBK, mt * kBM, bar);
    }
    if (g.b_mn) {
#pragma unroll
        for (int i = 0; i < (BN + 63) / 64; ++i) tma_load(sb + i * 8192, &g.b, nt * BN + i * 64, kb * kBK, bar);
    } else {
        tma_load(sb, &g.b, kb * kBK, nt * BN, bar);
    }
}

// The four products of a stage (16 contraction elements each).
__device__ __forceinline__ void mma_stage(const GemmArgs& g, const unsigned char* stage, uint32_t d, bool first)
{
    const uint64_t a = tile_desc(stage, g.a_mn), b = tile_desc(stage + kATile, g.b_mn);
    const uint64_t da = g.a_mn ? 2048 >> 4 : 32 >> 4, db = g.b_mn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
    for (int k = 0; k < kBK / 16; ++k) mma(d, a + k * da, b + k * db, g.idesc, !(first && k == 0));
}

__device__ __forceinline__ unsigned char* aligned_smem(unsigned char* p)
{
    return p + ((1024 - (smem_addr(p) & 1023)) & 1023);
}

// Tile t of the persistent order: columns of 16 m-tiles, so that the CTAs
// that run together share both operands in L2.
__device__ __forceinline__ void tile_at(const GemmArgs& g, int t, int* mt, int* nt)
{
    constexpr int kGroup = 16;
    const int per = kGroup * g.tiles_n, group = t / per, in = t - group * per;
    const int rows = min(kGroup, g.tiles_m - group * kGroup);
    *nt = in / rows;
    *mt = group * kGroup + in - *nt * rows;
}

// ---------------------------------------------------------------------------
// Many tiles: persistent CTAs
// ---------------------------------------------------------------------------

template <int BN, int STAGES>
__global__ void __launch_bounds__(kGemmThreads, 1) zero_gemm_kernel(const __grid_constant__ GemmArgs g)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = aligned_smem(raw);
    __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles = g.tiles_m * g.tiles_n;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int k = 0; k < 2; ++k) {
            mbar_init(&acc_full[k], 1);
            mbar_init(&acc_empty[k], 4);
        }
        mbar_init(&drained, 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async;" ::: "memory");
    }
    if (warp == 2) tmem_alloc(&tmem, 2 * BN);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t base = tmem;
    volatile int* abort = &abort_flag;

    if (warp == 0 && lane == 0) {
        int it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
            int mt, nt;
            tile_at(g, t, &mt, &nt);
            for (int kb = 0; kb < g.kblocks; ++kb, ++it) {
                const int s = it % STAGES;
                if (!wait(&empty[s], ((it / STAGES) & 1) ^ 1, abort)) {
                    ok = false;
                    break;
                }
                load_stage<BN>(g, smem + s * kStageBytes<BN>, &full[s], mt, nt, kb);
            }
        }
        // after a wait that ran out, the copies in flight land before the CTA ends
        if (!ok) {
            for (int k = max(0, it - STAGES); k < it; ++k) wait_landed(&full[k % STAGES], (k / STAGES) & 1);
        }
    } else if (warp == 1 && lane == 0) {
        int it = 0, n = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x, ++n) {
            const int acc = n & 1;
            ok = wait(&acc_empty[acc], ((n >> 1) & 1) ^ 1, abort);
            fence_after();
            for (int kb = 0; ok && kb < g.kblocks; ++kb, ++it) {
                const int s = it % STAGES;
                if (!wait(&full[s], (it / STAGES) & 1, abort)) {
                    ok = false;
                    break;
                }
                fence_after();
                mma_stage(g, smem + s * kStageBytes<BN>, base + acc * BN, kb == 0);
                mma_commit(&empty[s]);
            }
            if (ok) mma_commit(&acc_full[acc]);
        }
        if (!ok) { // products in flight end before the tensor memory goes
            mma_commit(&drained);
            wait_landed(&drained, 0);
        }
    } else if (warp >= 4) {
        const int q = warp & 3;
        int n = 0;
        for (int t = blockIdx.x; t < tiles; t += gridDim.x, ++n) {
            int mt, nt;
            tile_at(g, t, &mt, &nt);
            const int acc = n & 1;
            bool ok = wait(&acc_full[acc], (n >> 1) & 1, abort);
            if (!__all_sync(0xffffffffu, ok)) break;
            fence_after();
            const int row = mt * kBM + q * 32 + lane;
#pragma unroll 1
            for (int c = 0; c < BN; c += 32) {
                float v[32];
                tmem_load(base + acc * BN + c + (static_cast<uint32_t>(q * 32) << 16), v);
                if (row < g.m && nt * BN + c < g.n) emit32(g.o, row, nt * BN + c, v);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[acc]);
        }
    }
    __syncthreads();
    fence_after();
    if (warp == 2) tmem_free(base, 2 * BN);
}

// ---------------------------------------------------------------------------
// Few tiles: the contraction cut over a cluster
// ---------------------------------------------------------------------------

template <int BN, int STAGES>
__global__ void __launch_bounds__(kGemmThreads, 1) zero_gemm_split_kernel(const __grid_constant__ GemmArgs g)
{
    extern __shared__ unsigned char raw[];
    unsigned char* smem = aligned_smem(raw);
    __shared__ uint64_t full[STAGES], empty[STAGES], acc_full, drained;
    __shared__ uint32_t tmem;
    __shared__ int abort_flag;
    constexpr uint32_t kCols = BN < 32 ? 32 : BN;
    constexpr int kPitch = kBM + 1; // odd: rows and columns of the partial tile are both free of bank conflicts
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
    const int t = blockIdx.x / size;
    int mt, nt;
    tile_at(g, t, &mt, &nt);
    const int kb0 = static_cast<int>(static_cast<long long>(g.kblocks) * rank / size);
    const int kb1 = static_cast<int>(static_cast<long long>(g.kblocks) * (rank + 1) / size);
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

    if (warp == 0 && lane == 0) {
        int it = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const int s = it % STAGES;
            if (!wait(&empty[s], ((it / STAGES) & 1) ^ 1, abort)) {
                ok = false;
                break;
            }
            load_stage<BN>(g, smem + s * kStageBytes<BN>, &full[s], mt, nt, kb);
        }
        if (!ok) {
            for (int k = max(0, it - STAGES); k < it; ++k) wait_landed(&full[k % STAGES], (k / STAGES) & 1);
        }
    } else if (warp == 1 && lane == 0) {
        int it = 0;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
            const int s = it % STAGES;
            if (!wait(&full[s], (it / STAGES) & 1, abort)) {
                ok = false;
                break;
            }
            fence_after();
            mma_stage(g, smem + s * kStageBytes<BN>, base, kb == kb0);
            mma_commit(&empty[s]);
        }
        if (ok) {
            mma_commit(&acc_full);
        } else {
            mma_commit(&drained);
            wait_landed(&drained, 0);
        }
    }
    __syncwarp();
    // The stages are free once the last product is done: the partial tile goes
    // there, column by column.
    float* part = reinterpret_cast<float*>(smem);
    if (warp >= 4) {
        const int q = warp & 3;
        const bool ok = wait(&acc_full, 0, abort);
        if (__all_sync(0xffffffffu, ok)) {
            fence_after();
            const int row = q * 32 + lane;
            const uint32_t at = base + (static_cast<uint32_t>(q * 32) << 16);
            if constexpr (BN == 16) {
                float v[16];
                tmem_load16(at, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) part[j * kPitch + row] = v[j];
            } else {
#pragma unroll 1
                for (int c = 0; c < BN; c += 32) {
                    float v[32];
                    tmem_load(at + c, v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) part[(c + j) * kPitch + row] = v[j];
                }
            }
            fence_before();
        }
    }
    __syncwarp();
    cluster_sync();
    // Each CTA finishes a share of the tile: the partial sums of the cluster
    // are added in rank order.
    const int rows = min(kBM, g.m - mt * kBM), cols = min(BN, g.n - nt * BN);
    const uint32_t part_at = smem_addr(part);
    const int fast = g.o.swap ? rows : cols, total = rows * cols; // the output's contiguous index runs over lanes
    for (int e = rank * kGemmThreads + static_cast<int>(threadIdx.x); e < total; e += size * kGemmThreads) {
        const int hi = e / fast, lo = e - hi * fast;
        const int r = g.o.swap ? lo : hi, c = g.o.swap ? hi : lo;
        const uint32_t at = part_at + static_cast<uint32_t>(c * kPitch + r) * 4;
        float v = 0.0f;
        for (int k = 0; k < size; ++k) v += peer_load(at, static_cast<uint32_t>(k));
        const int gr = mt * kBM + r, gc = nt * BN + c;
        if (g.o.swap) emit(g.o, gc, gr, v);
        else emit(g.o, gr, gc, v);
    }
    cluster_sync(); // peers have read this CTA's part
    fence_after();
    if (warp == 2) tmem_free(base, kCols);
}

// ---------------------------------------------------------------------------
// dz = dy act'(z) and the sums of its columns; copies to aligned rows
// ---------------------------------------------------------------------------

constexpr int kSumCols = 256; // columns of a CTA: 32 lanes of 8

// Rows [chunk * rows_per, ...) of 256 columns: dz (where asked for) and the
// fp32 sum of each column over these rows.
__global__ void __launch_bounds__(256) zero_act_grad_kernel(const void* dy, long long lddy, const void* z, long long ldz,
                                                            void* dz, long long lddz, float* sums, long long T, int N,
                                                            int rows_per, int act, int bf16, int vec)
{
    const int lane = threadIdx.x & 31, line = threadIdx.x >> 5;
    const int col = blockIdx.x * kSumCols + lane * 8;
    const long long r0 = static_cast<long long>(blockIdx.y) * rows_per, r1 = min(T, r0 + rows_per);
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    if (vec && col + 8 <= N) {
#pragma unroll 4
        for (long long r = r0 + line; r < r1; r += 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(dy) + r * lddy + col);
            uint32_t g[4] = {u.x, u.y, u.z, u.w};
            if (act != ZERO_ACT_NONE) {
                const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(z) + r * ldz + col);
                const uint32_t h[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = unpack16(g[j], bf16), p = unpack16(h[j], bf16);
                    const float a = d.x * slope(p.x, act), b = d.y * slope(p.y, act);
                    sum[2 * j] += a;
                    sum[2 * j + 1] += b;
                    g[j] = pack16(a, b, bf16);
                }
                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dz) + r * lddz + col) = make_uint4(g[0], g[1], g[2], g[3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 d = unpack16(g[j], bf16);
                    sum[2 * j] += d.x;
                    sum[2 * j + 1] += d.y;
                }
            }
        }
    } else {
        for (long long r = r0 + line; r < r1; r += 8)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (col + j >= N) continue;
                float d = load16(dy, r * lddy + col + j, bf16);
                if (act != ZERO_ACT_NONE) {
                    d *= slope(load16(z, r * ldz + col + j, bf16), act);
                    store16(dz, r * lddz + col + j, d, bf16);
                }
                sum[j] += d;
            }
    }
    if (!sums) return;
    __shared__ float part[8][kSumCols];
#pragma unroll
    for (int j = 0; j < 8; ++j) part[line][lane * 8 + j] = sum[j];
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += part[k][threadIdx.x];
    const int c = blockIdx.x * kSumCols + threadIdx.x;
    if (c < N) sums[static_cast<long long>(blockIdx.y) * N + c] = s;
}

__global__ void __launch_bounds__(256) zero_bias_grad_kernel(const float* sums, int chunks, int N, void* db, int bf16)
{
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= N) return;
    float s = 0.0f;
    for (int k = 0; k < chunks; ++k) s += sums[static_cast<long long>(k) * N + c];
    store16(db, c, s, bf16);
}

// Rows that do not start on 16 bytes, laid out so that they do (a tensor map
// needs it).
__global__ void __launch_bounds__(256) zero_align_rows_kernel(const uint16_t* src, long long lds, uint16_t* dst,
                                                              long long ldd, long long rows, int cols)
{
    for (long long r = blockIdx.y; r < rows; r += gridDim.y)
        for (int c = blockIdx.x * 256 + threadIdx.x; c < cols; c += gridDim.x * 256) dst[r * ldd + c] = src[r * lds + c];
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

int make_map(CUtensorMap* map, const Matrix& x, int box_rows)
{
    EncodeFn encode = tensor_map_encoder();
    if (!encode) return zero_record_cuda_error(static_cast<int>(cudaErrorNotSupported));
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(x.cols), static_cast<cuuint64_t>(x.rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(x.ld) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, step[2] = {1, 1};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(x.p), dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
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

// Dynamic shared memory above 48 KB is allowed once per kernel and device.
int allow_smem(GemmKernel fn, int bytes, int cluster)
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
    if (e == cudaSuccess && cluster) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return record(e);
    if (n_known < 64) known[n_known++] = {dev, fn};
    return ZERO_OK;
}

template <int BN> constexpr int kSplitStages = BN >= 256 ? 4 : BN >= 128 ? 6 : 8;
template <int BN> constexpr int kSplitSmem = kSplitStages<BN> * kStageBytes<BN> + 1024;

struct Choice {
    GemmKernel fn;
    int bn, smem;
};

Choice pick_split(int bn)
{
    switch (bn) {
    case 16: return {zero_gemm_split_kernel<16, kSplitStages<16>>, 16, kSplitSmem<16>};
    case 32: return {zero_gemm_split_kernel<32, kSplitStages<32>>, 32, kSplitSmem<32>};
    case 64: return {zero_gemm_split_kernel<64, kSplitStages<64>>, 64, kSplitSmem<64>};
    default: return {zero_gemm_split_kernel<128, kSplitStages<128>>, 128, kSplitSmem<128>};
    }
}

// D[m, n] = sum_k A B with A = a (or its transpose, a_mn) and B likewise.
// Extents are below 2^31 - 256 (checked by the callers).
int gemm(const Matrix& a, int a_mn, const Matrix& b, int b_mn, int64_t k, Out o, int type, cudaStream_t stream)
{
    int sms = 0;
    int rc = sm_count(&sms);
    if (rc) return rc;
    GemmArgs g{};
    const int64_t m = a_mn ? a.cols : a.rows, n = b_mn ? b.cols : b.rows;
    g.m = static_cast<int>(m);
    g.n = static_cast<int>(n);
    g.kblocks = static_cast<int>((k + kBK - 1) / kBK);
    g.a_mn = a_mn;
    g.b_mn = b_mn;
    o.bf16 = type == ZERO_TYPE_BF16;
    g.o = o;
    g.tiles_m = static_cast<int>((m + kBM - 1) / kBM);

    // Few tiles leave SMs without work: below one big tile per SM the tiles
    // get smaller and the contraction is cut over a cluster.
    const int64_t big = g.tiles_m * ((n + 255) / 256);
    const bool split = big < sms;
    int bn = 256, parts = 1;
    if (split) {
        bn = 128;
        if (!b_mn)
            while (bn > 16 && n <= bn / 2) bn /= 2;
        else if (n <= 64) bn = 64;
        const int64_t tiles = g.tiles_m * ((n + bn - 1) / bn);
        while (parts < 8 && tiles * parts * 2 <= 2 * sms && g.kblocks >= parts * 4) parts *= 2;
    }
    g.tiles_n = static_cast<int>((n + bn - 1) / bn);
    const int64_t tiles = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
    if (tiles * parts > INT32_MAX) return ZERO_EINVAL;
    const unsigned int t = type == ZERO_TYPE_BF16 ? 1 : 0;
    g.idesc = (1u << 4) | (t << 7) | (t << 10) | (static_cast<unsigned int>(a_mn) << 15) |
              (static_cast<unsigned int>(b_mn) << 16) | (static_cast<unsigned int>(bn >> 3) << 17) | ((kBM >> 4) << 24);
    rc = make_map(&g.a, a, a_mn ? 64 : kBM);
    if (rc) return rc;
    rc = make_map(&g.b, b, b_mn ? 64 : bn);
    if (rc) return rc;

    if (!split) {
        constexpr int kStages = 4, kSmem = kStages * kStageBytes<256> + 1024;
        GemmKernel fn = zero_gemm_kernel<256, kStages>;
        rc = allow_smem(fn, kSmem, 0);
        if (rc) return rc;
        fn<<<static_cast<unsigned int>(std::min<int64_t>(tiles, sms)), kGemmThreads, kSmem, stream>>>(g);
        return record(cudaGetLastError());
    }
    const Choice c = pick_split(bn);
    rc = allow_smem(c.fn, c.smem, 1);
    if (rc) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned int>(tiles * parts));
    cfg.blockDim = dim3(kGemmThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(c.smem);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned int>(parts);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return record(cudaLaunchKernelEx(&cfg, c.fn, g));
}

bool aligned16(const void* p, int64_t ld) { return addr(p) % 16 == 0 && ld % 8 == 0; }

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

constexpr int64_t kMostExtent = INT32_MAX - 512;
constexpr int64_t kMostElements = int64_t{1} << 48; // of one matrix: far above any memory, so that no size overflows

bool bad_sizes(int64_t T, int64_t K, int64_t N, int32_t act, int32_t type)
{
    return T < 0 || T > kMostExtent || K < 1 || K > kMostExtent || N < 1 || N > kMostExtent ||
           std::max(T * std::max(K, N), N * K) > kMostElements || act < ZERO_ACT_NONE || act > ZERO_ACT_SILU ||
           (type != ZERO_TYPE_FP16 && type != ZERO_TYPE_BF16);
}

constexpr int64_t kMostLd = int64_t{1} << 38;

bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > kMostLd; }

// Rows of a chunk of the column sums: about four CTAs per SM, at least 32 rows.
int sum_rows(int64_t T, int64_t N)
{
    const int64_t stripes = (N + kSumCols - 1) / kSumCols;
    const int64_t want = std::max<int64_t>(1, 608 / stripes);
    return static_cast<int>(std::max<int64_t>(32, up((T + want - 1) / want, 8)));
}

int64_t sum_chunks(int64_t T, int64_t N)
{
    const int64_t r = sum_rows(T, N);
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

int align_rows(Matrix* x, void* to, cudaStream_t stream)
{
    const int64_t ld = up(x->cols, 8);
    const dim3 grid(static_cast<unsigned int>(std::min<int64_t>(8, (x->cols + 255) / 256)),
                    static_cast<unsigned int>(std::min<int64_t>(x->rows, 16384)));
    zero_align_rows_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x->p), x->ld, static_cast<uint16_t*>(to), ld,
                                                     x->rows, static_cast<int>(x->cols));
    x->p = to;
    x->ld = ld;
    return record(cudaGetLastError());
}

} // namespace

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
        c.take(sum_chunks(T, N) * N * 4);
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
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    int rc = ZERO_OK;
    if (fix_x && (rc = align_rows(&mx, tx, st))) return rc;
    if (fix_w && (rc = align_rows(&mw, tw, st))) return rc;
    Out o{};
    o.y = y, o.ldy = ldy, o.z = z, o.ldz = ldz, o.bias = bias, o.res = residual, o.ldr = ldr;
    o.rows = static_cast<int>(T), o.cols = static_cast<int>(N), o.act = act;
    o.vec = aligned16(y, ldy) && (!z || aligned16(z, ldz)) && (!residual || aligned16(residual, ldr)) && addr(bias) % 16 == 0;
    if (T <= 128) {
        o.swap = 1;
        return gemm(mw, 0, mx, 0, K, o, type, st);
    }
    return gemm(mx, 0, mw, 0, K, o, type, st);
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
    const bool fix_dy = products && !has_act && !aligned16(dy, lddy);
    Carver c{static_cast<unsigned char*>(workspace)};
    void* tx = fix_x ? c.take(matrix_bytes(T, K)) : nullptr;
    void* tw = fix_w ? c.take(matrix_bytes(N, K)) : nullptr;
    void* tz = has_act || fix_dy ? c.take(matrix_bytes(T, N)) : nullptr;
    const int64_t chunks = sum_chunks(T, N);
    float* sums = db ? static_cast<float*>(c.take(chunks * N * 4)) : nullptr;
    if (c.used > 0) {
        if (!workspace || workspace_bytes < c.used) return ZERO_EINVAL;
        if (addr(workspace) % 16) return ZERO_EALIGN;
    }
    Matrix mx{x, ldx, T, K}, mw{w, ldw, N, K}, mz{dy, lddy, T, N};
    int rc = ZERO_OK;
    const int bf16 = type == ZERO_TYPE_BF16;
    if (has_act || db) {
        const int vec = aligned16(dy, lddy) && (!has_act || aligned16(z, ldz));
        const int64_t ldt = up(N, 8);
        const dim3 grid(static_cast<unsigned int>((N + kSumCols - 1) / kSumCols), static_cast<unsigned int>(chunks));
        zero_act_grad_kernel<<<grid, 256, 0, st>>>(dy, lddy, z, ldz, has_act ? tz : nullptr, ldt, sums, T, static_cast<int>(N),
                                                   sum_rows(T, N), act, bf16, vec);
        if ((rc = record(cudaGetLastError()))) return rc;
        if (has_act) mz = {tz, ldt, T, N};
        if (db) {
            zero_bias_grad_kernel<<<static_cast<unsigned int>((N + 255) / 256), 256, 0, st>>>(sums, static_cast<int>(chunks),
                                                                                              static_cast<int>(N), db, bf16);
            if ((rc = record(cudaGetLastError()))) return rc;
        }
    }
    if (fix_dy && (rc = align_rows(&mz, tz, st))) return rc;
    if (fix_x && (rc = align_rows(&mx, tx, st))) return rc;
    if (fix_w && (rc = align_rows(&mw, tw, st))) return rc;
    if (dx) {
        Out o{};
        o.y = dx, o.ldy = lddx, o.rows = static_cast<int>(T), o.cols = static_cast<int>(K), o.vec = aligned16(dx, lddx);
        if (T <= 128) {
            o.swap = 1;
            rc = gemm(mw, 1, mz, 0, N, o, type, st);
        } else {
            rc = gemm(mz, 0, mw, 1, N, o, type, st);
        }
        if (rc) return rc;
    }
    if (dw) {
        Out o{};
        o.y = dw, o.ldy = lddw, o.rows = static_cast<int>(N), o.cols = static_cast<int>(K), o.vec = aligned16(dw, lddw);
        rc = gemm(mz, 1, mx, 1, T, o, type, st);
    }
    return rc;
}

extern "C" int zero_linear_timeouts(int64_t* count, int32_t reset)
{
    if (!count) return ZERO_EINVAL;
    unsigned int n = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&n, g_linear_timeouts, sizeof(n));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_linear_timeouts, &zero, sizeof(zero));
    }
    if (e != cudaSuccess) return record(e);
    *count = n;
    return ZERO_OK;
}
