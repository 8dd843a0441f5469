// The gated feed-forward projections h = act(x Wg^T + bg) * (x Wu^T + bu) and
// their gradients, on the 5th generation tensor cores of sm_103a (the kernels
// of gemm.cuh; linear.cu describes them).
//
// Forward: one launch, one product.  Half of a tile's columns are features of
// the gate, half the same features of the up projection: in a pair of CTAs each
// loads its half of that operand from its own matrix, so that every CTA's
// tensor memory ends up with both sums of an element and the epilogue writes
// h (and g and u where they are kept) without either passing through memory.
// The tokens' operand is read once for both.  With few tokens the operands
// change sides and the halves are rows.
//
// Backward, with g and u as the forward pass kept them:
//   du = dh act(g),  dg = dh u act'(g)        a pass over T x N, with the biases' column sums
//   dx = dg Wg + du Wu                        one product: dg and du lie side by side, its contraction
//                                             runs over Wg's features, then over Wu's
//   dWg = dg^T x,  dWu = du^T x
// All three products go into one launch where they take the same kernel.
//
// Bound by the tensor cores: x [8192, 2048], 8192 features, SiLU, bf16, g and u
// kept: forward 292 us (1880 TFLOP/s; 345 to 353 back to back at the card's power
// limit), the backward pass's products 605 us (1820 TFLOP/s, tensor pipe 97 %
// busy; in all 723 to 750, back to back 780 to 805).  With few tokens by the reads
// of the weights: 4 tokens 14 us (67 MB); backward, where the weights' gradients
// are written too (134 MB, 20 us at a copy's rate), 44: dg and du, dx and both dW
// are three launches, one after the other.
#include "gemm.cuh"

namespace {

// What has to be done before the products: dg and du side by side ([T][2
// half], zeros from N to half), their column sums over chunks of rows, and the
// copies of operands that do not lie on 16 bytes.
struct GatePrepArgs {
    const void* dh;
    const void* g;
    const void* u;
    void* dz;            // may be null
    float* sums;         // [chunks][2 N], may be null
    long long lddh, ldg, ldu, T;
    int N, half, rows_per, vec;
    int stripes, chunks;
    Copy copy[3];        // x, wg, wu
};

// dg and du are rounded to 16 bits here, once, as operands of the products;
// their column sums take them before that.
// Bound by HBM: it reads three elements and writes two for each of T x N (8192 x
// 8192 bf16, SiLU, 671 MB 107 us, 6270 GB/s; one, two or four rows of a thread in
// flight make no difference).
template <int ACT, int BF16>
__global__ void __launch_bounds__(256) zero_gated_prep_kernel(const __grid_constant__ GatePrepArgs a)
{
    let_successor_start();
    wait_for_predecessor();
    int cta = blockIdx.x - a.stripes * a.chunks;
    if (cta >= 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (cta >= 0 && cta < a.copy[k].ctas) copy_rows(a.copy[k], cta);
            cta -= a.copy[k].ctas;
        }
        return;
    }
    const int stripe = blockIdx.x % a.stripes, chunk = blockIdx.x / a.stripes;
    const int lane = threadIdx.x & 31, line = threadIdx.x >> 5;
    const int col = stripe * kSumCols + lane * 8;
    const long long r0 = static_cast<long long>(chunk) * a.rows_per, r1 = min(a.T, r0 + a.rows_per);
    const uint16_t* dh = static_cast<const uint16_t*>(a.dh);
    const uint16_t* g = static_cast<const uint16_t*>(a.g);
    const uint16_t* u = static_cast<const uint16_t*>(a.u);
    uint16_t* dz = static_cast<uint16_t*>(a.dz);
    float sg[8], su[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sg[j] = su[j] = 0.0f;
    auto through = [](float d, float gv, float uv, float* dg, float* du) {
        *du = d * activate<ACT>(gv);
        if constexpr (ACT == ZERO_ACT_RELU) *dg = gv > 0.0f ? d * uv : 0.0f;
        else *dg = d * (uv * slope<ACT>(gv)); // d u alone may leave the range that the slope brings it back to
    };
    const bool whole = a.vec && col + 8 <= a.N; // else by granules; zeros past the last feature
    if (col < a.half) {
#pragma unroll 2
        for (long long r = r0 + line; r < r1; r += 8) {
            const uint16_t *pd = dh + r * a.lddh, *pg = g + r * a.ldg, *pu = u + r * a.ldu;
            const uint4 d4 = whole ? *reinterpret_cast<const uint4*>(pd + col) : load_any(pd, col, a.N);
            const uint4 g4 = whole ? *reinterpret_cast<const uint4*>(pg + col) : load_any(pg, col, a.N);
            const uint4 u4 = whole ? *reinterpret_cast<const uint4*>(pu + col) : load_any(pu, col, a.N);
            const uint32_t dw[4] = {d4.x, d4.y, d4.z, d4.w}, gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
            uint32_t og[4], ou[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 d = unpack16(dw[j], BF16), gv = unpack16(gw[j], BF16), uv = unpack16(uw[j], BF16);
                float2 dg, du;
                through(d.x, gv.x, uv.x, &dg.x, &du.x);
                through(d.y, gv.y, uv.y, &dg.y, &du.y);
                sg[2 * j] += dg.x, sg[2 * j + 1] += dg.y;
                su[2 * j] += du.x, su[2 * j + 1] += du.y;
                og[j] = pack16(dg.x, dg.y, BF16);
                ou[j] = pack16(du.x, du.y, BF16);
            }
            if (dz) {
                *reinterpret_cast<uint4*>(dz + r * (2ll * a.half) + col) = make_uint4(og[0], og[1], og[2], og[3]);
                *reinterpret_cast<uint4*>(dz + r * (2ll * a.half) + a.half + col) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
            }
        }
    }
    if (!a.sums) return;
    __shared__ float part[8][kSumCols];
    const int c = stripe * kSumCols + threadIdx.x;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) part[line][lane * 8 + j] = k ? su[j] : sg[j];
        __syncthreads();
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += part[i][threadIdx.x];
        if (c < a.N) a.sums[static_cast<long long>(chunk) * 2 * a.N + k * static_cast<long long>(a.N) + c] = s;
    }
}

// The biases' gradients where no product follows to take them along.
__global__ void __launch_bounds__(32) zero_gated_bias_kernel(const __grid_constant__ GatedBackArgs args)
{
    wait_for_predecessor();
    bias_sum(args, threadIdx.x);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using GatePrepKernel = void (*)(GatePrepArgs);

GatePrepKernel pick_gate_prep(int act, int type)
{
    const bool b = type == ZERO_TYPE_BF16;
    switch (act) {
    case ZERO_ACT_RELU: return b ? zero_gated_prep_kernel<ZERO_ACT_RELU, 1> : zero_gated_prep_kernel<ZERO_ACT_RELU, 0>;
    case ZERO_ACT_GELU: return b ? zero_gated_prep_kernel<ZERO_ACT_GELU, 1> : zero_gated_prep_kernel<ZERO_ACT_GELU, 0>;
    case ZERO_ACT_SILU: return b ? zero_gated_prep_kernel<ZERO_ACT_SILU, 1> : zero_gated_prep_kernel<ZERO_ACT_SILU, 0>;
    default: return b ? zero_gated_prep_kernel<ZERO_ACT_NONE, 1> : zero_gated_prep_kernel<ZERO_ACT_NONE, 0>;
    }
}

// Where dg and du lie side by side, du starts on a block of the contraction.
int64_t half_of(int64_t N) { return up(N, kBK); }

// A product with its second weights and outputs.
struct GatedProduct {
    Product p;
    Matrix second;       // forward: the up projection's weights; dx: likewise
    const void* bias2;
    void* u;
    int64_t ldu;
    int64_t half;        // dx: blocks of the first part
};

// The product of the forward pass; few tokens change sides.
GatedProduct forward_product(const Matrix& x, const Matrix& wg, const Matrix& wu, const Out& o)
{
    GatedProduct q{};
    q.p = o.swap ? product(wg, 0, x, 0, o) : product(x, 0, wg, 0, o);
    q.p.twin = 1;
    q.second = wu;
    return q;
}

// dx = [dg du] [Wg; Wu].
GatedProduct dx_product(const Matrix& dz, const Matrix& wg, const Matrix& wu, const Out& o)
{
    GatedProduct q{};
    q.p = o.swap ? product(wg, 1, dz, 0, o) : product(dz, 0, wg, 1, o);
    q.p.k = dz.cols;
    q.second = wu;
    q.half = dz.cols / 2 / kBK;
    return q;
}

int fill(GatedProblem* g, const GatedProduct& q, const Variant& v, int type)
{
    const Product& p = q.p;
    const unsigned int t = type == ZERO_TYPE_BF16 ? 1 : 0;
    const bool twin = p.twin != 0;
    int bm = v.pair ? 256 : kBM, bn = v.bn;          // of a product's tile
    const int b_rows = v.pair ? v.bn / 2 : v.bn;
    g->o = p.o;
    g->bias2 = q.bias2;
    g->u_out = q.u;
    g->ldu = q.ldu;
    g->o.wide_y = widest_access(p.o.y, p.o.ldy);
    g->o.wide_z = widest_access(p.o.z, p.o.ldz);
    g->wide_u = widest_access(q.u, q.ldu);
    g->o.bf16 = type == ZERO_TYPE_BF16;
    g->a_mn = p.a_mn ? (p.a.cols % 64 == 0 ? 2 : 1) : 0;
    g->b_mn = p.b_mn ? (p.b.cols % 64 == 0 ? 2 : 1) : 0;
    g->m = static_cast<int>(p.m);
    g->n = static_cast<int>(p.n);
    g->idesc = (1u << 4) | (t << 7) | (t << 10) | (static_cast<unsigned int>(g->a_mn != 0) << 15) |
               (static_cast<unsigned int>(g->b_mn != 0) << 16) | (static_cast<unsigned int>(bn >> 3) << 17) |
               (static_cast<unsigned int>(bm >> 4) << 24);
    if (twin) (p.o.swap ? bm : bn) /= 2;
    g->tiles_m = static_cast<int>((p.m + bm - 1) / bm);
    g->tiles_n = static_cast<int>((p.n + bn - 1) / bn);
    g->kblocks = static_cast<int>(kblocks_of(p));
    g->cut = is_cut(p, v);
    g->half = static_cast<int>(q.half);
    g->second_a = q.half && p.o.swap;
    // boxes: in the forward pass half a tile's features at a time (a pair's CTAs load a half each anyway)
    const int a_box = twin && p.o.swap ? kBM / 2 : kBM, b_box = twin && !p.o.swap && !v.pair ? b_rows / 2 : b_rows;
    int rc;
    if ((rc = make_map(&g->a, p.a, g->a_mn, g->a_mn == 2 ? kBM / 64 : g->a_mn ? 64 : a_box))) return rc;
    if ((rc = make_map(&g->b, p.b, g->b_mn, g->b_mn == 2 ? b_rows / 64 : g->b_mn ? 64 : b_box))) return rc;
    if (q.second.p) {
        const bool a_side = p.o.swap;
        if ((rc = a_side ? make_map(&g->a2, q.second, g->a_mn, g->a_mn == 2 ? kBM / 64 : g->a_mn ? 64 : a_box)
                         : make_map(&g->b2, q.second, g->b_mn, g->b_mn == 2 ? b_rows / 64 : g->b_mn ? 64 : b_box)))
            return rc;
    }
    if (v.pair && p.o.vec) {
        if ((rc = make_map(&g->y, Matrix{p.o.y, p.o.ldy, p.m, p.n}, 0, 32))) return rc;
        if (p.o.z && (rc = make_map(&g->z, Matrix{p.o.z, p.o.ldz, p.m, p.n}, 0, 32))) return rc;
        if (q.u && (rc = make_map(&g->u, Matrix{q.u, q.ldu, p.m, p.n}, 0, 32))) return rc;
    }
    return ZERO_OK;
}

template <int COUNT, class Args>
int launch_gated(Args& args, int64_t clusters, const Variant& v, int sms, cudaStream_t stream)
{
    if (clusters * v.parts > INT32_MAX - 64) return ZERO_EINVAL;
    args.tiles = static_cast<int>(clusters);
    int rc;
    if (v.pair) {
        GemmKernel<Args> fn = zero_gemm_pair_kernel<256, kPairStages<256>, COUNT, Args>;
        if ((rc = allow_smem(reinterpret_cast<const void*>(fn), kPairSmem<256>))) return rc;
        return launch_after(fn, args, 2 * std::min<int64_t>(clusters, sms / 2), kGemmThreads, kPairSmem<256>, 2, stream);
    }
    const SplitPick<Args> k = pick_split<COUNT, Args>(v);
    if ((rc = allow_smem(reinterpret_cast<const void*>(k.fn), k.smem))) return rc;
    return launch_after(k.fn, args, clusters * v.parts, k.threads, k.smem, v.parts, stream);
}

struct GateSums {
    const float* sums;
    void* db;
    void* db2;
    int chunks, n;       // n: columns of a row of sums
};

// Up to three gradients' products in one launch.
int launch_backward(const GatedProduct* q, int count, int type, const GateSums* with, int sms, cudaStream_t stream)
{
    Product p[3];
    for (int k = 0; k < count; ++k) p[k] = q[k].p;
    double estimate;
    const Variant v = choose(p, count, sms, &estimate);
    GatedBackArgs args{};
    int64_t clusters = 0;
    for (int k = 0; k < count; ++k) {
        const int rc = fill(&args.p[k], q[k], v, type);
        if (rc) return rc;
        if (tiles_of(p[k], v) > INT32_MAX - 64) return ZERO_EINVAL;
        clusters += clusters_of(p[k], v);
        if (clusters * v.parts > INT32_MAX - 64) return ZERO_EINVAL;
        if (k < 2) args.ends[k] = static_cast<int>(clusters);
    }
    for (int k = count; k < 2; ++k) args.ends[k] = static_cast<int>(clusters);
    if (with) args.sums = with->sums, args.db = with->db, args.db2 = with->db2, args.chunks = with->chunks, args.n_db = with->n;
    args.bf16 = type == ZERO_TYPE_BF16;
    return launch_gated<3>(args, clusters, v, sms, stream);
}

// The gradients' products in the order they are launched in, and how many of
// them go into the first launch.
int first_launch(GatedProduct* q, int count, bool has_dx, int sms)
{
    if (!has_dx || count == 1) return count;
    Product p[3];
    for (int k = 0; k < count; ++k) p[k] = q[k].p;
    double one, first, second;
    choose(p, count, sms, &one);
    choose(p, 1, sms, &first);
    choose(p + 1, count - 1, sms, &second);
    if (first + second < one) return 1;
    // the longer tiles first
    if (kblocks_of(p[1]) > kblocks_of(p[0])) std::rotate(q, q + 1, q + count);
    return count;
}

bool bad_gated(int64_t T, int64_t K, int64_t N, int32_t act, int32_t type)
{
    return bad_sizes(T, K, N, act, type) || N > kMostExtent / 2 || 2 * T * N > kMostElements;
}

} // namespace

// The waits of this unit's kernels that ran out (zero_train_timeouts, linear.cu).
__attribute__((visibility("hidden"))) int zero_gated_wait_timeouts(unsigned int* count, int reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_gemm_timeouts, sizeof(*count));
    if (e == cudaSuccess && reset) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_gemm_timeouts, &zero, sizeof(zero));
    }
    return record(e);
}

extern "C" int zero_gated_workspace(int64_t T, int64_t K, int64_t N, int32_t backward, int32_t aligned, int64_t* bytes)
{
    if (!bytes || bad_gated(T, K, N, ZERO_ACT_NONE, ZERO_TYPE_FP16)) return ZERO_EINVAL;
    Carver c{nullptr};
    if (!aligned) {
        c.take(matrix_bytes(T, K));
        c.take(matrix_bytes(N, K));
        c.take(matrix_bytes(N, K));
    }
    if (backward) {
        c.take(T * 2 * half_of(N) * 2);
        c.take(sum_chunks(T, N, ZERO_ACT_NONE) * 2 * N * 4);
    }
    *bytes = c.used;
    return ZERO_OK;
}

extern "C" int zero_gated_plan(int64_t T, int64_t K, int64_t N, int32_t products, int32_t* launches, int32_t* rows, int32_t* columns,
                               int32_t* cluster, int32_t* per_sm)
{
    if (!launches || !rows || !columns || !cluster || !per_sm || products < 0 || products > 3 || T < 1 ||
        bad_gated(T, K, N, ZERO_ACT_NONE, ZERO_TYPE_FP16))
        return ZERO_EINVAL;
    int sms = 0;
    const int rc = sm_count(&sms);
    if (rc) return rc;
    const int64_t half = half_of(N);
    const Matrix x{nullptr, K, T, K}, w{nullptr, K, N, K}, dz{nullptr, 2 * half, T, 2 * half}, dg{nullptr, 2 * half, T, N};
    Out o{};
    o.swap = T <= kFewTokens;
    GatedProduct q[3];
    int count = 0;
    if (products == 0) q[count++] = forward_product(x, w, w, o);
    if (products & 1) q[count++] = dx_product(dz, w, w, o);
    o.swap = 0;
    for (int k = 0; k < 2 && (products & 2); ++k) q[count++].p = product(dg, 1, x, 1, o);
    const int first = first_launch(q, count, products & 1, sms);
    *launches = first < count ? 2 : 1;
    Product p[3];
    for (int k = 0; k < count; ++k) p[k] = q[k].p;
    double estimate;
    const Variant v = choose(p, first, sms, &estimate);
    *rows = v.pair ? 256 : kBM;
    *columns = v.bn;
    *cluster = v.pair ? 2 : v.parts;
    *per_sm = v.per_sm;
    return ZERO_OK;
}

extern "C" int zero_gated_forward(const void* x, int64_t ldx, const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, const void* bg,
                                  const void* bu, void* h, int64_t ldh, void* g, int64_t ldg, void* u, int64_t ldu, int64_t T, int64_t K,
                                  int64_t N, int32_t act, int32_t type, void* workspace, int64_t workspace_bytes, void* cuda_stream)
{
    if (bad_gated(T, K, N, act, type) || !g != !u) return ZERO_EINVAL;
    if (T == 0) return ZERO_OK;
    if (!x || !wg || !wu || !h || bad_ld(ldx, K) || bad_ld(ldwg, K) || bad_ld(ldwu, K) || bad_ld(ldh, N) || (g && bad_ld(ldg, N)) ||
        (u && bad_ld(ldu, N)))
        return ZERO_EINVAL;
    for (const void* p : {x, wg, wu, bg, bu, static_cast<const void*>(h), static_cast<const void*>(g), static_cast<const void*>(u)})
        if (addr(p) % 2) return ZERO_EALIGN;
    const Matrix in[] = {{x, ldx, T, K}, {wg, ldwg, N, K}, {wu, ldwu, N, K}, {bg, N, 1, N}, {bu, N, 1, N}},
                 out[] = {{h, ldh, T, N}, {g, ldg, T, N}, {u, ldu, T, N}};
    for (int i = 0; i < 3; ++i) {
        for (const Matrix& m : in)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, m.p, m.ld, m.rows, m.cols)) return ZERO_EOVERLAP;
        for (int j = i + 1; j < 3; ++j)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, out[j].p, out[j].ld, out[j].rows, out[j].cols)) return ZERO_EOVERLAP;
    }
    Matrix mx = in[0], mg = in[1], mu = in[2];
    Matrix* operands[] = {&mx, &mg, &mu};
    Carver c{static_cast<unsigned char*>(workspace)};
    void* to[3] = {};
    for (int k = 0; k < 3; ++k)
        if (!aligned16(operands[k]->p, operands[k]->ld)) to[k] = c.take(matrix_bytes(operands[k]->rows, operands[k]->cols));
    if (c.used > 0) {
        if (!workspace || workspace_bytes < c.used) return ZERO_EINVAL;
        if (addr(workspace) % 16) return ZERO_EALIGN;
        for (const Matrix& m : in)
            if (in_workspace(workspace, c.used, m.p, m.ld, m.rows, m.cols)) return ZERO_EOVERLAP;
        for (const Matrix& m : out)
            if (in_workspace(workspace, c.used, m.p, m.ld, m.rows, m.cols)) return ZERO_EOVERLAP;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    int rc = ZERO_OK, ctas = 0, sms = 0;
    GatePrepArgs prep{};
    for (int k = 0; k < 3; ++k)
        if (to[k]) add_copy(&prep.copy[k], &ctas, operands[k], to[k]);
    if (ctas && (rc = launch_after(pick_gate_prep(ZERO_ACT_NONE, type), prep, ctas, 256, 0, 1, st))) return rc;
    if ((rc = sm_count(&sms))) return rc;
    Out o{};
    o.y = h, o.ldy = ldh, o.z = g, o.ldz = ldg, o.bias = bg, o.act = act;
    o.vec = aligned16(h, ldh) && (!g || (aligned16(g, ldg) && aligned16(u, ldu))) && addr(bg) % 16 == 0 && addr(bu) % 16 == 0;
    o.swap = T <= kFewTokens;
    GatedProduct q = forward_product(mx, mg, mu, o);
    q.bias2 = bu, q.u = u, q.ldu = ldu;
    double estimate;
    const Variant v = choose(&q.p, 1, sms, &estimate);
    GatedArgs args{};
    if ((rc = fill(&args.p, q, v, type))) return rc;
    if (tiles_of(q.p, v) > INT32_MAX - 64) return ZERO_EINVAL;
    return launch_gated<1>(args, clusters_of(q.p, v), v, sms, st);
}

extern "C" int zero_gated_backward(const void* dh, int64_t lddh, const void* g, int64_t ldg, const void* u, int64_t ldu, const void* x,
                                   int64_t ldx, const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, void* dx, int64_t lddx, void* dwg,
                                   int64_t lddwg, void* dwu, int64_t lddwu, void* dbg, void* dbu, int64_t T, int64_t K, int64_t N, int32_t act,
                                   int32_t type, void* workspace, int64_t workspace_bytes, void* cuda_stream)
{
    if (bad_gated(T, K, N, act, type)) return ZERO_EINVAL;
    if (!dx && !dwg && !dwu && !dbg && !dbu) return ZERO_EINVAL;
    if ((dwg && bad_ld(lddwg, K)) || (dwu && bad_ld(lddwu, K))) return ZERO_EINVAL;
    const bool any_dw = dwg || dwu;
    if (T > 0 && (!dh || !g || !u || bad_ld(lddh, N) || bad_ld(ldg, N) || bad_ld(ldu, N) ||
                  (dx && (!wg || !wu || bad_ld(ldwg, K) || bad_ld(ldwu, K) || bad_ld(lddx, K))) || (any_dw && (!x || bad_ld(ldx, K)))))
        return ZERO_EINVAL;
    if (!dx) wg = wu = nullptr;
    if (!any_dw) x = nullptr;
    for (const void* p : {dh, g, u, x, wg, wu, static_cast<const void*>(dx), static_cast<const void*>(dwg), static_cast<const void*>(dwu),
                          static_cast<const void*>(dbg), static_cast<const void*>(dbu)})
        if (addr(p) % 2) return ZERO_EALIGN;
    const Matrix in[] = {{dh, lddh, T, N}, {g, ldg, T, N}, {u, ldu, T, N}, {x, ldx, T, K}, {wg, ldwg, N, K}, {wu, ldwu, N, K}},
                 out[] = {{dx, lddx, T, K}, {dwg, lddwg, N, K}, {dwu, lddwu, N, K}, {dbg, N, 1, N}, {dbu, N, 1, N}};
    for (int i = 0; i < 5; ++i) {
        for (const Matrix& m : in)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, m.p, m.ld, m.rows, m.cols)) return ZERO_EOVERLAP;
        for (int j = i + 1; j < 5; ++j)
            if (share(out[i].p, out[i].ld, out[i].rows, out[i].cols, out[j].p, out[j].ld, out[j].rows, out[j].cols)) return ZERO_EOVERLAP;
    }
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (T == 0) { // sums over no tokens
        cudaError_t e = cudaSuccess;
        for (int k = 1; k < 5 && e == cudaSuccess; ++k)
            if (out[k].p)
                e = cudaMemset2DAsync(const_cast<void*>(out[k].p), static_cast<size_t>(out[k].ld) * 2, 0, static_cast<size_t>(out[k].cols) * 2,
                                      static_cast<size_t>(out[k].rows), st);
        return record(e);
    }
    const bool products = dx || any_dw, bias = dbg || dbu;
    const int64_t half = half_of(N);
    Matrix mx = in[3], mg = in[4], mu = in[5];
    Matrix* operands[] = {&mx, &mg, &mu};
    Carver c{static_cast<unsigned char*>(workspace)};
    void* to[3] = {};
    for (int k = 0; k < 3; ++k)
        if (operands[k]->p && !aligned16(operands[k]->p, operands[k]->ld)) to[k] = c.take(matrix_bytes(operands[k]->rows, operands[k]->cols));
    uint16_t* dz = products ? static_cast<uint16_t*>(c.take(T * 2 * half * 2)) : nullptr;
    const int64_t chunks = sum_chunks(T, N, ZERO_ACT_NONE);
    float* sums = bias ? static_cast<float*>(c.take(chunks * 2 * N * 4)) : nullptr;
    if (!workspace || workspace_bytes < c.used) return ZERO_EINVAL;
    if (addr(workspace) % 16) return ZERO_EALIGN;
    for (const Matrix& m : in)
        if (in_workspace(workspace, c.used, m.p, m.ld, m.rows, m.cols)) return ZERO_EOVERLAP;
    for (const Matrix& m : out)
        if (in_workspace(workspace, c.used, m.p, m.ld, m.rows, m.cols)) return ZERO_EOVERLAP;

    GatePrepArgs prep{};
    prep.dh = dh, prep.g = g, prep.u = u, prep.dz = dz, prep.sums = sums, prep.lddh = lddh, prep.ldg = ldg, prep.ldu = ldu, prep.T = T;
    prep.N = static_cast<int>(N), prep.half = static_cast<int>(half), prep.rows_per = sum_rows(T, N, ZERO_ACT_NONE);
    prep.vec = aligned16(dh, lddh) && aligned16(g, ldg) && aligned16(u, ldu);
    prep.stripes = static_cast<int>((N + kSumCols - 1) / kSumCols); // half is below the last stripe's end
    prep.chunks = static_cast<int>(chunks);
    if (chunks * prep.stripes > INT32_MAX - 3 * 4864) return ZERO_EINVAL;
    int rc = ZERO_OK, ctas = prep.stripes * prep.chunks, sms = 0;
    for (int k = 0; k < 3; ++k)
        if (to[k]) add_copy(&prep.copy[k], &ctas, operands[k], to[k]);
    if ((rc = launch_after(pick_gate_prep(act, type), prep, ctas, 256, 0, 1, st))) return rc;

    const GateSums gate_sums{sums, dbg, dbu, static_cast<int>(chunks), static_cast<int>(2 * N)};
    if (!products) {
        GatedBackArgs args{};
        args.sums = sums, args.db = dbg, args.db2 = dbu, args.chunks = gate_sums.chunks, args.n_db = gate_sums.n, args.bf16 = type == ZERO_TYPE_BF16;
        return launch_after(zero_gated_bias_kernel, args, (2 * N + 31) / 32, 32, 0, 1, st);
    }
    const GateSums* with = bias ? &gate_sums : nullptr;
    if ((rc = sm_count(&sms))) return rc;
    GatedProduct q[3];
    int count = 0;
    if (dx) {
        Out o{};
        o.y = dx, o.ldy = lddx, o.vec = aligned16(dx, lddx), o.swap = T <= kFewTokens;
        q[count++] = dx_product(Matrix{dz, 2 * half, T, 2 * half}, mg, mu, o);
    }
    for (int k = 0; k < 2; ++k) {
        void* dw = k ? dwu : dwg;
        if (!dw) continue;
        Out o{};
        o.y = dw, o.ldy = k ? lddwu : lddwg, o.vec = aligned16(dw, o.ldy);
        q[count] = GatedProduct{};
        q[count++].p = product(Matrix{dz + k * half, 2 * half, T, N}, 1, mx, 1, o);
    }
    const int first = first_launch(q, count, dx != nullptr, sms);
    if ((rc = launch_backward(q, first, type, with, sms, st))) return rc;
    return first < count ? launch_backward(q + first, count - first, type, nullptr, sms, st) : ZERO_OK;
}
