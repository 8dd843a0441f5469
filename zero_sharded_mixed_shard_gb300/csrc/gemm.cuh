// Products of 16-bit operands on the 5th generation tensor cores of sm_103a,
// D[m, n] = sum_k A[m, k] B[n, k] with fp32 accumulators in tensor memory, and
// their epilogues: shared by the linear layer and the gated projections.
// linear.cu describes the two kernels.
#pragma once

#include <cuda.h> // driver types only: the tensor-map encoder is found through the runtime

#include <cmath>
#include <type_traits>
#include <utility>

#include "layers.cuh"

namespace {

constexpr int kGemmThreads = 384; // warp 0 TMA, warp 1 MMA, warp 2 tensor memory, warp 3 bias sums, warps 4..11 epilogue
constexpr int kEpilogueWarps = 8;
constexpr int kBM = 128;          // rows of a tile: the lanes of tensor memory
constexpr int kBK = 64;           // contraction per stage: 128 bytes, one swizzle row
constexpr int kATile = kBM * kBK * 2;
constexpr unsigned long long kWaitLimitNs = 2000000000ull;

__device__ unsigned int g_gemm_timeouts;

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
    static constexpr int kTwin = 0;
};

// The gated projections.  Forward (kTwin 1): one product whose tile holds as
// many columns (swapped: rows) of the gate as of the up projection, so that
// both meet in one epilogue.  Backward (kTwin 2): dx, whose contraction runs
// over the gate's features and then over the up projection's, and both dW.
struct GatedProblem : Problem {
    CUtensorMap a2, b2;  // forward: the up projection's weights; dx: those of the second part
    CUtensorMap u;       // forward, pairs, where o.vec: like y and z (which holds the gate)
    const void* bias2;
    void* u_out;
    long long ldu;
    int wide_u;
    int half;            // dx: blocks of the contraction in its first part, else 0
    int second_a;        // dx: the operand of two parts is A
};

struct GatedArgs {
    GatedProblem p;
    int tiles;
    static constexpr int kTwin = 1;
};

struct GatedBackArgs {
    GatedProblem p[3];
    int ends[2];         // tiles (clusters) up to the end of the first and of the second product
    int tiles;
    const float* sums;   // [chunks][n_db]: the gate's columns, then the up projection's
    void* db;
    void* db2;           // either may be null
    int chunks, n_db, bf16;
    static constexpr int kTwin = 2;
};

// The product that tile (cluster) t belongs to, and its place among that
// product's.
template <int COUNT> __device__ __forceinline__ const Problem& problem_of(const GemmArgs& args, int t, int* at)
{
    const bool second = COUNT == 2 && t >= args.tiles0;
    *at = t - (second ? args.tiles0 : 0);
    return args.p[COUNT == 1 ? 0 : second];
}

template <int COUNT> __device__ __forceinline__ const GatedProblem& problem_of(const GatedArgs& args, int t, int* at)
{
    *at = t;
    return args.p;
}

template <int COUNT> __device__ __forceinline__ const GatedProblem& problem_of(const GatedBackArgs& args, int t, int* at)
{
    const int k = t < args.ends[0] ? 0 : t < args.ends[1] ? 1 : 2;
    *at = t - (k ? args.ends[k - 1] : 0);
    return args.p[k];
}

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

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
    if (atomicExch(const_cast<int*>(abort), 1) == 0) atomicAdd(&g_gemm_timeouts, 1u);
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

// GELU in tanh's form is z s(u), u = 2 sqrt(2 / pi) (z + 0.044715 z^3), and
// SiLU z s(z), with s the logistic function 1 / (1 + 2^(-x log2 e)).
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

__device__ __forceinline__ void bias_sum(const GatedArgs&, int) {}

// Both biases' gradients, one after the other in a row of sums.
__device__ __forceinline__ void bias_sum(const GatedBackArgs& args, int lane)
{
    const int n = args.n_db / 2;
    for (long long c = blockIdx.x * 32ll + lane; c < args.n_db; c += gridDim.x * 32ll) {
        float s = 0.0f;
#pragma unroll 16
        for (int k = 0; k < args.chunks; ++k) s += args.sums[static_cast<long long>(k) * args.n_db + c];
        void* db = c < n ? args.db : args.db2;
        if (db) store16(db, c < n ? c : c - n, s, args.bf16);
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

// The gated projections' results: h = act(g) u, and g and u themselves where
// they are kept.  One element, and eight neighbours.
__device__ __forceinline__ void emit_gated(const GatedProblem& p, long long row, int col, float g, float u)
{
    const Out& o = p.o;
    if (o.bias) g += load16(o.bias, col, o.bf16);
    if (p.bias2) u += load16(p.bias2, col, o.bf16);
    if (o.z) {
        store16(o.z, row * o.ldz + col, g, o.bf16);
        store16(p.u_out, row * p.ldu + col, u, o.bf16);
    }
    float v[1] = {g};
    activate_all(v, o.act);
    store16(o.y, row * o.ldy + col, v[0] * u, o.bf16);
}

__device__ __forceinline__ void emit_gated8(const GatedProblem& p, long long row, int col, float (&g)[8], float (&u)[8])
{
    const Out& o = p.o;
    if (o.bias) add8(g, __ldg(reinterpret_cast<const uint4*>(at16(o.bias, 0, 0, col))), o.bf16);
    if (p.bias2) add8(u, __ldg(reinterpret_cast<const uint4*>(at16(p.bias2, 0, 0, col))), o.bf16);
    if (o.z) {
        *reinterpret_cast<uint4*>(at16(o.z, o.ldz, row, col)) = pack8(g, o.bf16);
        *reinterpret_cast<uint4*>(at16(p.u_out, p.ldu, row, col)) = pack8(u, o.bf16);
    }
    activate_all(g, o.act);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= u[j];
    *reinterpret_cast<uint4*>(at16(o.y, o.ldy, row, col)) = pack8(g, o.bf16);
}

template <int BF16> __device__ __forceinline__ void add_bias_any(const void* bias, int vec, int col, int cols, float (&v)[32], int lane)
{
    if (!bias) return;
    if (vec && cols == 32) {
        const uint4* b = reinterpret_cast<const uint4*>(at16(bias, 0, 0, col));
#pragma unroll
        for (int q = 0; q < 4; ++q) add8(v + 8 * q, __ldg(b + q), BF16);
        return;
    }
    const float mine = lane < cols ? load16(bias, col + lane, BF16) : 0.0f;
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] += __shfl_sync(0xffffffffu, mine, j);
}

// 32 x 32 results of a warp, lane l holding row row0 + l.
template <int BF16>
__device__ __forceinline__ void emit_gated_piece_as(const GatedProblem& p, long long row0, int rows, int col0, int cols, float (&g)[32],
                                                    float (&u)[32], uint4* piece, int lane)
{
    const Out& o = p.o;
    add_bias_any<BF16>(o.bias, o.vec, col0, cols, g, lane);
    add_bias_any<BF16>(p.bias2, o.vec, col0, cols, u, lane);
    auto put = [&](const float(&v)[32], void* to, long long ld, int wide) {
        piece_row(piece, v, BF16, lane);
        __syncwarp();
        piece_out(piece, at16(to, ld, row0, col0), ld, rows, cols, wide, lane);
        __syncwarp();
    };
    if (o.z) {
        put(g, o.z, o.ldz, o.wide_z);
        put(u, p.u_out, p.ldu, p.wide_u);
    }
    activate_all(g, o.act);
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] *= u[j];
    put(g, o.y, o.ldy, o.wide_y);
}

__device__ __forceinline__ void emit_gated_piece(const GatedProblem& p, long long row0, int rows, int col0, int cols, float (&g)[32],
                                                 float (&u)[32], uint4* piece, int lane)
{
    if (p.o.bf16) emit_gated_piece_as<1>(p, row0, rows, col0, cols, g, u, piece, lane);
    else emit_gated_piece_as<0>(p, row0, rows, col0, cols, g, u, piece, lane);
}

// 32 rows x 64 columns of a pair's tile, whole ones by TMA stores: the gate's
// accumulators at `acc`, the up projection's BN / 2 columns on.  What is kept
// is written first, each from the staging that the last store has left.
template <int BN, int BF16, class Release>
__device__ __forceinline__ void emit_gated_whole(const GatedProblem& p, uint32_t acc, int row0, int col, uint4* staging, int lane, Release release)
{
    const Out& o = p.o;
    if (o.z) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) { // the gate, then the up projection
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                float v[32];
                tmem_load(acc + k * (BN / 2) + h * 32, v);
                add_bias_any<BF16>(k ? p.bias2 : o.bias, 1, col + h * 32, 32, v, lane);
                if (h == 0) staging_free();
                stage_row<BF16>(staging, h, v, lane);
            }
            send_staging(k ? &p.u : &p.z, col, row0, staging);
        }
    }
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        float g[32], u[32];
        tmem_load(acc + h * 32, g);
        tmem_load(acc + BN / 2 + h * 32, u);
        if (h == 1) release();
        add_bias_any<BF16>(o.bias, 1, col + h * 32, 32, g, lane);
        add_bias_any<BF16>(p.bias2, 1, col + h * 32, 32, u, lane);
        activate_all(g, o.act);
#pragma unroll
        for (int j = 0; j < 32; ++j) g[j] *= u[j];
        if (h == 0) staging_free();
        stage_row<BF16>(staging, h, g, lane);
    }
    send_staging(&p.y, col, row0, staging);
}

template <int BN, class Release>
__device__ __forceinline__ void emit_gated_block(const GatedProblem& p, uint32_t acc, int row0, int rows, int col, uint4* staging, int lane,
                                                 Release release)
{
    if (p.o.vec && rows > 0 && col + 64 <= p.n) {
        if (p.o.bf16) emit_gated_whole<BN, 1>(p, acc, row0, col, staging, lane, release);
        else emit_gated_whole<BN, 0>(p, acc, row0, col, staging, lane, release);
        return;
    }
    staging_free();
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        const int cols = min(32, p.n - (col + h * 32));
        if (rows > 0 && cols > 0) {
            float g[32], u[32];
            tmem_load(acc + h * 32, g);
            tmem_load(acc + BN / 2 + h * 32, u);
            emit_gated_piece(p, row0, rows, col + h * 32, cols, g, u, staging, lane);
        }
    }
    release();
}

template <int BN, int STAGES, int COUNT, class Args>
__global__ void __launch_bounds__(kGemmThreads, 1) zero_gemm_pair_kernel(const __grid_constant__ Args args)
{
    constexpr int kTwin = Args::kTwin;
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
            int at, mt, nt;
            const auto& g = problem_of<COUNT>(args, t, &at);
            tile_at(g, at, &mt, &nt);
            // a tile of the gated projections has half of its columns from either of them, a CTA's half each
            const int m0 = mt * 256 + rank * kBM, n0 = kTwin == 1 ? nt * (BN / 2) : nt * BN + rank * (BN / 2);
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
                const CUtensorMap* map_b = &g.b;
                int k = kb * kBK; // of B: the weights' two parts start at their own 0, dz has them side by side
                if constexpr (kTwin == 1) {
                    if (rank) map_b = &g.b2;
                } else if constexpr (kTwin == 2) {
                    if (g.half && kb >= g.half) map_b = &g.b2, k -= g.half * kBK;
                }
                if (g.a_mn == 2) {
                    tma_load_pair3(sa, &g.a, kb * kBK, m0 / 64, bar);
                } else if (g.a_mn) {
                    tma_load_pair(sa, &g.a, m0, kb * kBK, bar);
                    tma_load_pair(sa + 8192, &g.a, m0 + 64, kb * kBK, bar);
                } else {
                    tma_load_pair(sa, &g.a, kb * kBK, m0, bar);
                }
                if (g.b_mn == 2) {
                    tma_load_pair3(sb, map_b, k, n0 / 64, bar);
                } else if (g.b_mn) {
#pragma unroll
                    for (int i = 0; i < BN / 128; ++i) tma_load_pair(sb + i * 8192, map_b, n0 + i * 64, k, bar);
                } else {
                    tma_load_pair(sb, map_b, k, n0, bar);
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
            int at;
            const auto& g = problem_of<COUNT>(args, t, &at);
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
            int place, mt, nt;
            const auto& g = problem_of<COUNT>(args, t, &place);
            tile_at(g, place, &mt, &nt);
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
            if constexpr (kTwin == 1) {
                // columns [64 h, 64 h + 64) of both halves, h = 0, 1
                const int c = c0 / 2;
                emit_gated_block<BN>(g, base + acc * BN + c + (static_cast<uint32_t>(q * 32) << 16), row0, rows, nt * (BN / 2) + c, staging,
                                     lane, release);
            }
#pragma unroll 1
            for (int c = kTwin == 1 ? c0 + BN / 2 : c0; c < c0 + BN / 2; c += 64) {
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

// The same for the gated projections, whose two sums of an element lie `up`
// floats apart in a partial tile.
template <int PARTS> __device__ __forceinline__ void join_gated(const GatedProblem& p, const Join& j, int up)
{
    const int vecs = p.o.vec ? j.fast / 8 : 0;
    for (int e = j.self; e < vecs * j.slow; e += j.everyone) {
        const int s = e / vecs, f = (e - s * vecs) * 8;
        const uint32_t at = j.part + static_cast<uint32_t>(s * j.pitch + f) * 4;
        float g[8], u[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) g[h] = u[h] = 0.0f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float4 a = peer_load4(at + h * 16, j.first + k), b = peer_load4(at + up * 4 + h * 16, j.first + k);
                g[4 * h] += a.x, g[4 * h + 1] += a.y, g[4 * h + 2] += a.z, g[4 * h + 3] += a.w;
                u[4 * h] += b.x, u[4 * h + 1] += b.y, u[4 * h + 2] += b.z, u[4 * h + 3] += b.w;
            }
        }
        emit_gated8(p, j.row0 + s, j.col0 + f, g, u);
    }
    const int left = j.fast - vecs * 8;
    for (int e = j.self; e < left * j.slow; e += j.everyone) {
        const int s = e / left, f = e - s * left + vecs * 8;
        const uint32_t at = j.part + static_cast<uint32_t>(s * j.pitch + f) * 4;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            g += peer_load(at, j.first + k);
            u += peer_load(at + up * 4, j.first + k);
        }
        emit_gated(p, j.row0 + s, j.col0 + f, g, u);
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

template <int BN, int PER_SM, int COUNT, class Args>
__global__ void __launch_bounds__((kSplitThreads<BN, PER_SM>), PER_SM) zero_gemm_split_kernel(const __grid_constant__ Args args)
{
    constexpr int kTwin = Args::kTwin;
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
    int at;
    const auto& g = problem_of<COUNT>(args, cluster, &at);
    const int t = g.cut ? at : at * size + rank;
    // extents of a tile in the output: half of the gated projections' features
    const int tile_m = kTwin == 1 && g.o.swap ? kBM / 2 : kBM, tile_n = kTwin == 1 && !g.o.swap ? BN / 2 : BN;
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
            if constexpr (kTwin == 1) { // the gate's features and the up projection's in one operand
                tma_load(sa, &g.a, kb * kBK, mt * tile_m, &full[s]);
                if (g.o.swap) tma_load(sa + kATile / 2, &g.a2, kb * kBK, mt * tile_m, &full[s]);
                tma_load(sb, &g.b, kb * kBK, nt * tile_n, &full[s]);
                if (!g.o.swap) tma_load(sb + BN / 2 * kBK * 2, &g.b2, kb * kBK, nt * tile_n, &full[s]);
                continue;
            }
            const CUtensorMap *map_a = &g.a, *map_b = &g.b;
            int ka = kb * kBK, kbb = kb * kBK;
            if constexpr (kTwin == 2) { // the weights' second part starts at its own 0
                if (g.half && kb >= g.half) {
                    if (g.second_a) map_a = &g.a2, ka -= g.half * kBK;
                    else map_b = &g.b2, kbb -= g.half * kBK;
                }
            }
            if (g.a_mn == 2) {
                tma_load3(sa, map_a, ka, mt * (kBM / 64), &full[s]);
            } else if (g.a_mn) {
                tma_load(sa, map_a, mt * kBM, ka, &full[s]);
                tma_load(sa + 8192, map_a, mt * kBM + 64, ka, &full[s]);
            } else {
                tma_load(sa, map_a, ka, mt * kBM, &full[s]);
            }
            if (BN >= 64 && g.b_mn == 2) {
                tma_load3(sb, map_b, kbb, nt * (BN / 64), &full[s]);
            } else if (BN >= 64 && g.b_mn) {
#pragma unroll
                for (int i = 0; i < BN / 64; ++i) tma_load(sb + i * 8192, map_b, nt * BN + i * 64, kbb, &full[s]);
            } else {
                tma_load(sb, map_b, kbb, nt * BN, &full[s]);
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
    const int rows = idle ? 0 : min(tile_m, g.m - mt * tile_m), cols = min(tile_n, g.n - nt * tile_n);
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
            if constexpr (kTwin == 1 && BN >= 64) {
                if (direct) { // 32 columns of both at a time
#pragma unroll 1
                    for (int c = ((warp - 4) >> 2) * 32; c < BN / 2; c += kThreads == 384 ? 64 : 32) {
                        if (q * 32 >= rows || c >= cols) continue;
                        float v[32], u[32];
                        tmem_load(acc + c, v);
                        tmem_load(acc + BN / 2 + c, u);
                        emit_gated_piece(g, mt * kBM + q * 32, min(32, rows - q * 32), nt * tile_n + c, min(32, cols - c), v, u,
                                         reinterpret_cast<uint4*>(smem + (warp - 4) * kPieceBytes), lane);
                    }
                }
            }
#pragma unroll 1
            for (int c = kTwin == 1 && direct ? BN : c0; c < c0 + kSpan; c += kStep) {
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
        j.row0 = o.swap ? nt * tile_n : mt * tile_m;
        j.col0 = o.swap ? mt * tile_m : nt * tile_n;
        j.first = g.cut ? 0 : static_cast<uint32_t>(rank);
        j.self = (g.cut ? rank * kThreads : 0) + static_cast<int>(threadIdx.x);
        j.everyone = (g.cut ? size : 1) * kThreads;
        if constexpr (kTwin == 1) {
            const int up = o.swap ? kBM / 2 : BN / 2; // from the gate's to the up projection's, in floats
            switch (parts) {
            case 1: join_gated<1>(g, j, up); break;
            case 2: join_gated<2>(g, j, up); break;
            case 4: join_gated<4>(g, j, up); break;
            default: join_gated<8>(g, j, up); break;
            }
        } else {
            switch (parts) {
            case 1: join<1>(o, j); break;
            case 2: join<2>(o, j); break;
            case 4: join<4>(o, j); break;
            default: join<8>(o, j); break;
            }
        }
    }
    cluster_sync(); // peers have read this CTA's part
    fence_after();
    if (warp == 2) tmem_free(base, kCols);
}

// ---------------------------------------------------------------------------
// Copies to rows on 16 bytes
// ---------------------------------------------------------------------------

// A matrix whose rows do not start on 16 bytes, laid out so that they do (a
// tensor map needs it).
struct Copy {
    const uint16_t* src;
    uint16_t* dst;
    long long lds, ldd, rows;
    int cols, ctas;
};

// 8 elements a thread, two bytes at a time (four-byte reads where rows allow
// them were no faster, nor whole granules shifted: the copies' time is latency,
// and of large ones their writes').
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

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn tensor_map_encoder()
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
inline int make_map(CUtensorMap* map, const Matrix& x, int mn, int extent)
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

template <class Args> using GemmKernel = void (*)(Args);

template <int BN> constexpr int kPairStages = BN >= 256 ? 6 : 8;

template <int BN> constexpr int kPairSmem = kPairStages<BN> * kPairStage<BN> + kEpilogueBytes + 1024;

// A product to be launched: D[m, n] = sum_k A[m, k] B[n, k].
struct Product {
    Matrix a, b;
    int a_mn, b_mn;
    int64_t m, n, k;
    Out o;
    int twin;            // the gated projections: a tile's features are half of the one's, half of the other's
};

inline Product product(const Matrix& a, int a_mn, const Matrix& b, int b_mn, const Out& o)
{
    return {a, b, a_mn, b_mn, a_mn ? a.cols : a.rows, b_mn ? b.cols : b.rows, a_mn ? a.rows : a.cols, o, 0};
}

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

inline int64_t tiles_of(const Product& p, const Variant& v)
{
    int64_t bm = v.pair ? 256 : kBM, bn = v.bn;
    if (p.twin) (p.o.swap ? bm : bn) /= 2;
    return ((p.m + bm - 1) / bm) * ((p.n + bn - 1) / bn);
}

inline int64_t kblocks_of(const Product& p) { return (p.k + kBK - 1) / kBK; }

// Whether a cluster of v.parts CTAs shares a tile's contraction; one with
// fewer than two blocks a CTA is left whole.
inline bool is_cut(const Product& p, const Variant& v) { return v.parts > 1 && kblocks_of(p) >= 2 * v.parts; }

inline int64_t clusters_of(const Product& p, const Variant& v)
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
inline Variant choose(const Product* p, int count, int sms, double* estimate)
{
    // a tile has no more columns than the widest product needs; an MN-major operand comes in blocks of 64
    int widest = 16;
    bool swapped = false;
    for (int k = 0; k < count; ++k) {
        int bn = p[k].b_mn ? 64 : 16;
        while (bn < 128 && bn < (p[k].twin && !p[k].o.swap ? 2 * p[k].n : p[k].n)) bn *= 2;
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

// The split kernel of a variant.
template <class Args> struct SplitPick {
    GemmKernel<Args> fn;
    int smem, threads;
};

template <int COUNT, class Args> SplitPick<Args> pick_split(const Variant& v)
{
    auto pick = [](auto columns, auto per_sm) -> SplitPick<Args> {
        constexpr int BN = decltype(columns)::value, PER = decltype(per_sm)::value;
        return {zero_gemm_split_kernel<BN, PER, COUNT, Args>, kSplitSmem<BN, PER>, kSplitThreads<BN, PER>};
    };
    using std::integral_constant;
    if (v.bn == 16) return pick(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    if (v.bn == 32) return pick(integral_constant<int, 32>{}, integral_constant<int, 2>{});
    if (v.bn == 64 && v.per_sm == 2) return pick(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    if (v.bn == 64) return pick(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    return pick(integral_constant<int, 128>{}, integral_constant<int, 1>{});
}

// Up to this many tokens a tile's rows are features (y) or inputs (dx), its columns tokens.
constexpr int64_t kFewTokens = 128;

constexpr int kSumCols = 256; // columns of a CTA: 32 lanes of 8

// Rows of a chunk of the column sums: four CTAs per SM, five (all that fit)
// where an activation's arithmetic wants the warps, and at least 8 rows.
inline int sum_rows(int64_t T, int64_t N, int act)
{
    const int64_t stripes = (N + kSumCols - 1) / kSumCols;
    const int64_t want = std::max<int64_t>(1, (act == ZERO_ACT_NONE ? 608 : 760) / stripes);
    return static_cast<int>(std::max<int64_t>(8, up((T + want - 1) / want, 8)));
}

inline int64_t sum_chunks(int64_t T, int64_t N, int act)
{
    const int64_t r = sum_rows(T, N, act);
    return std::max<int64_t>(1, (T + r - 1) / r);
}

// Adds the copy of x to rows on 16 bytes to a launch of the preparing kernel.
inline void add_copy(Copy* to_do, int* ctas, Matrix* x, void* to)
{
    const int64_t ld = up(x->cols, 8), vecs = x->rows * (ld / 8);
    Copy& c = *to_do;
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
