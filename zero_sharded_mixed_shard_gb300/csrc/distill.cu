// The loss of a language model's logits against target tokens and against a
// teacher's top logits, and its gradient, in one launch.
//
// For a row s of V logits, its target g, and the teacher's K logits r_k at the
// indices j_k (z = temperature, a = alpha, w = the row's weight):
//   q = softmax(s), q' = softmax(s / z) over V,   p = softmax(r / z) over K
//   loss = w ((1 - a) (-log q_g) + a z^2 sum_k p_k (log p_k - log q'_{j_k}))
//   ds_j = w c ((1 - a) (q_j - [j = g]) + a z (q'_j - sum_{k: j_k = j} p_k))
// with c the call's gradient scale (p's sum is 1, so that the teacher's part
// of ds is z times a difference of two distributions).
//
// A CTA takes a row.  One pass over it finds the largest logit and the sums of
// exponentials (each thread's own largest so far, joined at the end), a second
// one writes the gradient; the second reads the row from L2.  Both sums share
// the largest logit, since it is the same for s / z.  The gradient's few
// elements at the target and the indices are written last, after the CTA's
// barrier, from logits read before the second pass: logits and gradient may be
// one matrix.
#include "layers.cuh"

namespace {

constexpr int kLossThreads = 512;
constexpr int kLossWarps = kLossThreads / 32;
constexpr int kMostTeacher = 1024; // entries of a row's teacher

struct LossArgs {
    const void* logits;
    const int32_t* targets;
    const int32_t* index;
    const void* teacher;
    const float* weights;
    float* loss;
    void* grad;          // null: the loss alone
    long long ldl, ldk, ldg;
    int V, K, teacher_type;
    float hard, soft;    // 1 - alpha, alpha
    float z, scale;
};

__device__ __forceinline__ float teacher_at(const void* p, long long i, int type)
{
    if (type == ZERO_TYPE_FP32) return static_cast<const float*>(p)[i];
    return load16(p, i, type == ZERO_TYPE_BF16);
}

// Sums of exponentials held with the largest value: sum 2^(l (x - top)).
struct Tops {
    float top, sum, soft;
};

// x - top without the difference of two infinities of one sign.
__device__ __forceinline__ float below(float x, float top) { return top == -INFINITY ? x : x - top; }

__device__ __forceinline__ Tops join(const Tops& p, const Tops& q, float l, float lz)
{
    Tops o;
    o.top = fmaxf(p.top, q.top);
    const float dp = p.top == o.top ? 0.0f : p.top - o.top, dq = q.top == o.top ? 0.0f : q.top - o.top;
    o.sum = p.sum * fast_exp2(dp * l) + q.sum * fast_exp2(dq * l);
    o.soft = p.soft * fast_exp2(dp * lz) + q.soft * fast_exp2(dq * lz);
    return o;
}

__device__ __forceinline__ float block_sum(float v, float* part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < kLossWarps; ++k) s += part[k];
    return s;
}

__device__ __forceinline__ float block_max(float v, float* part)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = part[0];
#pragma unroll
    for (int k = 1; k < kLossWarps; ++k) s = fmaxf(s, part[k]);
    return s;
}

__device__ __forceinline__ void widen8(const uint4& u, float (&v)[8], int bf16)
{
    const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = unpack16(h[j], bf16);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}

// VEC: a row of the gradient starts as far from a boundary of 16 bytes as its
// row of logits.  BOTH: two sums at different temperatures; otherwise one that
// serves the term in use (or both, at temperature 1).
template <int BF16, int VEC, int BOTH>
__global__ void __launch_bounds__(kLossThreads) zero_distill_kernel(const __grid_constant__ LossArgs a)
{
    __shared__ float part[kLossWarps];
    __shared__ Tops tops[kLossWarps];
    __shared__ float p_of[kMostTeacher], s_of[kMostTeacher];
    __shared__ int j_of[kMostTeacher];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* s = static_cast<const uint16_t*>(a.logits) + row * a.ldl;
    uint16_t* ds = static_cast<uint16_t*>(a.grad) + (a.grad ? row * a.ldg : 0);
    const float w = a.weights ? a.weights[row] : 1.0f;
    const int target = a.targets ? a.targets[row] : -1;
    const bool hard = a.hard != 0.0f && w != 0.0f && target >= 0 && target < a.V;

    // the teacher's distribution
    bool soft = a.soft != 0.0f && w != 0.0f && a.K > 0;
    float entropy = 0.0f; // sum p log p
    if (soft) {
        float top = -INFINITY, bad = 0.0f;
        for (int k = tid; k < a.K; k += kLossThreads) {
            const int j = a.index[row * a.ldk + k];
            const bool in = j >= 0 && j < a.V;
            const float r = in ? teacher_at(a.teacher, row * a.ldk + k, a.teacher_type) : -INFINITY;
            j_of[k] = in ? j : -1;
            p_of[k] = r;
            s_of[k] = in ? load16(s, j, BF16) : 0.0f;
            top = fmaxf(top, r);
            if (r != r) bad = 1.0f;
        }
        top = block_max(top, part);
        bad = block_max(bad, part);
        soft = top != -INFINITY || bad != 0.0f; // some entry has a probability
        float sum = 0.0f;
        for (int k = tid; k < a.K; k += kLossThreads) sum += j_of[k] < 0 ? 0.0f : expf((p_of[k] - top) / a.z);
        sum = block_sum(sum, part);
        const float log_sum = logf(sum);
        float h = 0.0f;
        for (int k = tid; k < a.K; k += kLossThreads) {
            const float d = (p_of[k] - top) / a.z, p = j_of[k] < 0 ? 0.0f : expf(d) / sum;
            if (p != 0.0f) h += p * (d - log_sum); // NaN goes on
            p_of[k] = p;
        }
        entropy = block_sum(h, part);
    }
    // the row's vectors lie in [head, rest); without them everything is rest
    const int head = VEC ? min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(s) & 15)) & 15) / 2) : 0;
    const int rest = VEC ? head + (a.V - head) / 8 * 8 : 0;
    const float s_target = hard ? load16(s, target, BF16) : 0.0f;

    if (!hard && !soft) { // nothing to learn from this row, whatever it holds
        if (tid == 0) a.loss[row] = 0.0f;
        if (a.grad) {
            for (int c = head + tid * 8; c < rest; c += kLossThreads * 8) *reinterpret_cast<uint4*>(ds + c) = make_uint4(0, 0, 0, 0);
            if (tid < head) ds[tid] = 0;
            for (int c = rest + tid; c < a.V; c += kLossThreads) ds[c] = 0;
        }
        return;
    }

    // the largest logit and the sums
    const float l1 = kLog2e, lz = kLog2e / a.z;
    const float l = BOTH || hard ? l1 : lz; // not BOTH: the one that is in use
    Tops mine = {-INFINITY, 0.0f, 0.0f};
    auto take = [&](const float (&v)[8]) {
        float top = v[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) top = fmaxf(top, v[j]);
        if (top > mine.top) {
            const float d = mine.top - top;
            mine.sum *= fast_exp2(d * l);
            if (BOTH) mine.soft *= fast_exp2(d * lz);
            mine.top = top;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = below(v[j], mine.top);
            mine.sum += fast_exp2(d * l);
            if (BOTH) mine.soft += fast_exp2(d * lz);
        }
    };
    if (VEC) {
#pragma unroll 4
        for (int c = head + tid * 8; c < rest; c += kLossThreads * 8) {
            float v[8];
            widen8(*reinterpret_cast<const uint4*>(s + c), v, BF16);
            take(v);
        }
    }
    // what lies before and behind the vectors: fewer than 16 elements where there are any
    for (int c = tid < head ? tid : rest + tid - head; c < a.V; c += kLossThreads * 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = c + j * kLossThreads;
            v[j] = at < a.V && (j == 0 || !VEC) ? load16(s, at, BF16) : -INFINITY;
        }
        take(v);
        if (VEC) break;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Tops other;
        other.top = __shfl_xor_sync(0xffffffffu, mine.top, o);
        other.sum = __shfl_xor_sync(0xffffffffu, mine.sum, o);
        other.soft = __shfl_xor_sync(0xffffffffu, mine.soft, o);
        mine = join(mine, other, l, lz);
    }
    if (lane == 0) tops[warp] = mine;
    __syncthreads();
    Tops all = tops[0];
#pragma unroll
    for (int k = 1; k < kLossWarps; ++k) all = join(all, tops[k], l, lz);
    const float sum_hard = all.sum, sum_soft = BOTH ? all.soft : all.sum;

    // the loss
    float cross = 0.0f; // sum p log q'
    if (soft) {
        float h = 0.0f;
        const float log_sum = logf(sum_soft);
        for (int k = tid; k < a.K; k += kLossThreads) {
            const float p = p_of[k];
            if (p != 0.0f) h += p * ((s_of[k] - all.top) / a.z - log_sum);
        }
        cross = block_sum(h, part);
    }
    if (tid == 0) {
        float v = 0.0f;
        if (hard) v += a.hard * (logf(sum_hard) - (s_target - all.top));
        if (soft) v += a.soft * a.z * a.z * (entropy - cross);
        a.loss[row] = w * v;
    }
    if (!a.grad) return;

    // the gradient: f_hard 2^(l1 (s - top)) + f_soft 2^(lz (s - top))
    const float g = w * a.scale;
    const float f_hard = hard ? g * a.hard / sum_hard : 0.0f, f_soft = soft ? g * a.soft * a.z / sum_soft : 0.0f;
    const float f_one = f_hard + f_soft;
    auto slope = [&](float x) {
        const float d = below(x, all.top);
        if (BOTH) return fmaf(f_hard, fast_exp2(d * l1), f_soft * fast_exp2(d * lz));
        return f_one * fast_exp2(d * l);
    };
    if (VEC) {
#pragma unroll 4
        for (int c = head + tid * 8; c < rest; c += kLossThreads * 8) {
            float v[8];
            widen8(*reinterpret_cast<const uint4*>(s + c), v, BF16);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = slope(v[j]);
            *reinterpret_cast<uint4*>(ds + c) = pack8(v, BF16);
        }
        if (tid < head) store16(ds, tid, slope(load16(s, tid, BF16)), BF16);
    }
#pragma unroll 8
    for (int c = rest + tid; c < a.V; c += kLossThreads) store16(ds, c, slope(load16(s, c, BF16)), BF16);
    __syncthreads(); // every element has its sum's part
    const float g_soft = g * a.soft * a.z;
    if (soft) {
        for (int k = tid; k < a.K; k += kLossThreads) {
            const int j = j_of[k];
            if (j < 0) continue;
            float p = 0.0f; // an index that occurs twice: each writes the same whole value
            for (int i = 0; i < a.K; ++i)
                if (j_of[i] == j) p += p_of[i];
            float v = slope(s_of[k]) - g_soft * p;
            if (hard && j == target) v -= g * a.hard;
            store16(ds, j, v, BF16);
        }
    }
    if (hard && tid == 0) {
        bool listed = false;
        if (soft)
            for (int i = 0; i < a.K; ++i) listed = listed || j_of[i] == target;
        if (!listed) store16(ds, target, slope(s_target) - g * a.hard, BF16);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using LossKernel = void (*)(LossArgs);

template <int BF16> LossKernel pick_loss(bool vec, bool both)
{
    if (vec) return both ? zero_distill_kernel<BF16, 1, 1> : zero_distill_kernel<BF16, 1, 0>;
    return both ? zero_distill_kernel<BF16, 0, 1> : zero_distill_kernel<BF16, 0, 0>;
}

// A matrix for share(), which counts in 16 bits.
struct Extent {
    const void* p;
    int64_t ld, rows, cols;
};

Extent extent(const void* p, int64_t ld, int64_t rows, int64_t cols, int64_t size) { return {p, ld * size / 2, rows, cols * size / 2}; }

bool meet(const Extent& p, const Extent& q) { return share(p.p, p.ld, p.rows, p.cols, q.p, q.ld, q.rows, q.cols); }

} // namespace

extern "C" int zero_distill_loss(const void* logits, int64_t ldl, const int32_t* targets, const int32_t* index, const void* teacher,
                                 int64_t ldk, const float* weights, float* loss, void* dlogits, int64_t lddl, int64_t T, int64_t V,
                                 int64_t K, float temperature, float alpha, float grad_scale, int32_t type, int32_t teacher_type,
                                 void* cuda_stream)
{
    if (T < 0 || T > kMostExtent || V < 1 || V > (int64_t{1} << 30) || K < 0 || K > kMostTeacher || T * V > kMostElements ||
        !(temperature >= 0.0009765625f && temperature <= 1024.0f) || !(alpha >= 0.0f && alpha <= 1.0f) ||
        !(grad_scale > -INFINITY && grad_scale < INFINITY) || (type != ZERO_TYPE_FP16 && type != ZERO_TYPE_BF16))
        return ZERO_EINVAL;
    if (alpha == 0.0f) K = 0; // the teacher is not looked at
    if (K > 0 && teacher_type != ZERO_TYPE_FP16 && teacher_type != ZERO_TYPE_BF16 && teacher_type != ZERO_TYPE_FP32) return ZERO_EINVAL;
    if (T == 0) return ZERO_OK;
    if (!logits || !loss || bad_ld(ldl, V) || (dlogits && bad_ld(lddl, V)) || (alpha < 1.0f && !targets) ||
        (K > 0 && (!index || !teacher || bad_ld(ldk, K))))
        return ZERO_EINVAL;
    if (alpha == 1.0f) targets = nullptr;
    if (K == 0) index = nullptr, teacher = nullptr;
    const int64_t size = teacher_type == ZERO_TYPE_FP32 ? 4 : 2;
    if (addr(logits) % 2 || addr(dlogits) % 2 || addr(targets) % 4 || addr(index) % 4 || addr(teacher) % size || addr(weights) % 4 ||
        addr(loss) % 4)
        return ZERO_EALIGN;
    const Extent in[] = {extent(logits, ldl, T, V, 2), extent(targets, T, 1, T, 4), extent(index, ldk, T, K, 4), extent(teacher, ldk, T, K, size),
                         extent(weights, T, 1, T, 4)},
                 out[] = {extent(loss, T, 1, T, 4), extent(dlogits, lddl, T, V, 2)};
    if (meet(out[0], out[1])) return ZERO_EOVERLAP;
    for (const Extent& o : out)
        for (const Extent& i : in) {
            const bool in_place = &o == &out[1] && &i == &in[0] && dlogits == logits && lddl == ldl;
            if (!in_place && meet(o, i)) return ZERO_EOVERLAP;
        }
    LossArgs a{};
    a.logits = logits, a.targets = targets, a.index = index, a.teacher = teacher, a.weights = weights, a.loss = loss, a.grad = dlogits;
    a.ldl = ldl, a.ldk = ldk, a.ldg = lddl, a.V = static_cast<int>(V), a.K = static_cast<int>(K), a.teacher_type = teacher_type;
    a.hard = 1.0f - alpha, a.soft = alpha, a.z = temperature, a.scale = grad_scale;
    const bool both = alpha > 0.0f && alpha < 1.0f && K > 0 && temperature != 1.0f;
    // every row of the gradient starts as far from a boundary of 16 bytes as that of the logits
    const bool vec = !dlogits || ((addr(logits) - addr(dlogits)) % 16 == 0 && (ldl - lddl) % 8 == 0);
    return launch_after(type == ZERO_TYPE_BF16 ? pick_loss<1>(vec, both) : pick_loss<0>(vec, both), a, T, kLossThreads, 0, 1,
                        static_cast<cudaStream_t>(cuda_stream));
}
