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
#include "gemm.cuh"

// Defined in adamw.cu (not exported): the step's part of zero_train_timeouts.
__attribute__((visibility("hidden"))) int zero_adamw_wait_timeouts(unsigned int* count, int reset);
// Defined in gated.cu (not exported): the gated projections' part.
__attribute__((visibility("hidden"))) int zero_gated_wait_timeouts(unsigned int* count, int reset);

namespace {

// ---------------------------------------------------------------------------
// dz = dy act'(z) and the sums of its columns; copies to aligned rows
// ---------------------------------------------------------------------------

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
        GemmKernel<GemmArgs> fn = count == 1 ? zero_gemm_pair_kernel<256, kPairStages<256>, 1, GemmArgs>
                                             : zero_gemm_pair_kernel<256, kPairStages<256>, 2, GemmArgs>;
        if ((rc = allow_smem(reinterpret_cast<const void*>(fn), kPairSmem<256>))) return rc;
        return launch_after(fn, args, 2 * std::min<int64_t>(tiles, sms / 2), kGemmThreads, kPairSmem<256>, 2, stream);
    }
    const SplitPick<GemmArgs> k = count == 1 ? pick_split<1, GemmArgs>(v) : pick_split<2, GemmArgs>(v);
    if ((rc = allow_smem(reinterpret_cast<const void*>(k.fn), k.smem))) return rc;
    return launch_after(k.fn, args, tiles * v.parts, k.threads, k.smem, v.parts, stream);
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
    if (fix_x) add_copy(&prep.copy[0], &ctas, &mx, tx);
    if (fix_w) add_copy(&prep.copy[1], &ctas, &mw, tw);
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
    if (fix_x) add_copy(&prep.copy[0], &ctas, &mx, tx);
    if (fix_w) add_copy(&prep.copy[1], &ctas, &mw, tw);
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
    cudaError_t e = cudaMemcpyFromSymbol(&n, g_gemm_timeouts, sizeof(n));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_gemm_timeouts, &zero, sizeof(zero));
    }
    if (e != cudaSuccess) return record(e);
    unsigned int steps = 0, gated = 0;
    int rc = zero_adamw_wait_timeouts(&steps, reset);
    if (!rc) rc = zero_gated_wait_timeouts(&gated, reset);
    if (rc) return rc;
    *count = static_cast<int64_t>(n) + steps + gated;
    return ZERO_OK;
}
