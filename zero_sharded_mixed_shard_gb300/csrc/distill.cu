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
// the largest logit, since it is the same for s / z.  One warp stays out of
// both passes where there is a teacher: its distribution, the loss, and the
// gradient's elements at the target and the indices are that warp's, and are
// stored last, after the CTA's barrier, from logits read before the second
// pass: logits and gradient may be one matrix.
// Bound by HBM and, nearly, by issue and exponentials: 8192 rows of 44629 bf16
// logits with 64 of a teacher's at temperature 2 (1.47 GB) 275 us, 5330 GB/s;
// without a teacher 260 us, the loss alone 146 and 131.  (Each block's barrier for
// the teacher's sums, scalar arithmetic and two exponentials an element 466 us.)
#include "layers.cuh"

namespace {

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

__device__ __forceinline__ Tops join(const Tops& p, const Tops& q, float l, float lz)
{
    Tops o;
    o.top = fmaxf(p.top, q.top);
    const float dp = p.top == o.top ? 0.0f : p.top - o.top, dq = q.top == o.top ? 0.0f : q.top - o.top;
    o.sum = p.sum * fast_exp2(dp * l) + q.sum * fast_exp2(dq * l);
    o.soft = p.soft * fast_exp2(dp * lz) + q.soft * fast_exp2(dq * lz);
    return o;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float2 exp2_2(float2 a) { return make_float2(fast_exp2(a.x), fast_exp2(a.y)); }

// The larger of each half; a NaN loses.
template <int BF16> __device__ __forceinline__ uint32_t max16(uint32_t a, uint32_t b)
{
    if constexpr (BF16) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    } else {
        const __half2 m = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
}

// The exponentials of two logits below the largest: `hard` 2^(l d), `soft`
// 2^(lz d).  SUMS 0: one serves both (in `hard`).  1: two of them.  2 and 4: the
// temperature is that, and e^d is a power of e^(d / z): half of the
// exponentials (8192 rows of 44629 with 64 of a teacher's at temperature 2 or 4
// 280 to 283 us, with two of them 293, as at temperatures 1.5 and 3; 9133 of 10007
// 86 to 90, 94; 16384 of 1000 60, 62).
template <int SUMS> __device__ __forceinline__ void exponentials(float2 d, float l, float lz, float2* hard, float2* soft)
{
    if constexpr (SUMS == 0) {
        *hard = exp2_2(mul2(d, make_float2(l, l)));
        return;
    }
    *soft = exp2_2(mul2(d, make_float2(lz, lz)));
    if constexpr (SUMS == 1) {
        *hard = exp2_2(mul2(d, make_float2(l, l)));
    } else {
        *hard = mul2(*soft, *soft);
        if constexpr (SUMS == 4) *hard = mul2(*hard, *hard);
    }
}

constexpr int kAtOnce = 4;         // vectors of a thread in flight
constexpr int kFewTeachers = 256;  // up to these the teacher's warp merges its entries alone

// VEC: a row of the gradient starts as far from a boundary of 16 bytes as its
// row of logits.
template <int BF16, int VEC, int SUMS, int kLossThreads>
__global__ void __launch_bounds__(kLossThreads, kLossThreads == 64 ? 20 : kLossThreads == 128 ? 10 : 4) zero_distill_kernel(const __grid_constant__ LossArgs a)
{
    constexpr int kLossWarps = kLossThreads / 32;
    __shared__ Tops tops[kLossWarps];
    // the teacher's entries: probabilities, logits at their indices, the gradient's values, the indices
    extern __shared__ float entries[];
    float *p_of = entries, *s_of = p_of + a.K, *v_of = s_of + a.K;
    int* j_of = reinterpret_cast<int*>(v_of + a.K);
    __shared__ int soft_flag;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long row = blockIdx.x;
    let_successor_start();
    wait_for_predecessor();
    const uint16_t* s = static_cast<const uint16_t*>(a.logits) + row * a.ldl;
    uint16_t* ds = static_cast<uint16_t*>(a.grad) + (a.grad ? row * a.ldg : 0);
    const float w = a.weights ? a.weights[row] : 1.0f;
    const int target = a.targets ? a.targets[row] : -1;
    const bool hard = a.hard != 0.0f && w != 0.0f && target >= 0 && target < a.V;
    const bool teacher = a.soft != 0.0f && w != 0.0f && a.K > 0;
    // the row's vectors lie in [head, rest); without them everything is rest
    const int head = VEC ? min(a.V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(s) & 15)) & 15) / 2) : 0;
    const int rest = VEC ? head + (a.V - head) / 8 * 8 : 0;
    const float s_target = hard ? load16(s, target, BF16) : 0.0f;
    const float l1 = kLog2e, lz = kLog2e / a.z;
    const float l = SUMS || hard ? l1 : lz; // one sum: the temperature of the term in use
    // the threads that go over the row
    const int self = teacher ? tid - 32 : tid, everyone = teacher ? kLossThreads - 32 : kLossThreads;

    Tops mine = {-INFINITY, 0.0f, 0.0f};
    float entropy = 0.0f; // sum p log p
    if (self < 0) {
        // the teacher's distribution
        float top = -INFINITY, bad = 0.0f;
        for (int k = lane; k < a.K; k += 32) {
            const int j = a.index[row * a.ldk + k];
            const bool in = j >= 0 && j < a.V;
            const float r = in ? teacher_at(a.teacher, row * a.ldk + k, a.teacher_type) : -INFINITY;
            j_of[k] = in ? j : -1;
            p_of[k] = r;
            s_of[k] = in ? load16(s, j, BF16) : 0.0f;
            top = fmaxf(top, r);
            if (r != r) bad = 1.0f;
        }
        top = warp_max(top);
        bad = warp_max(bad);
        float sum = 0.0f;
        for (int k = lane; k < a.K; k += 32) sum += j_of[k] < 0 ? 0.0f : expf((p_of[k] - top) / a.z);
        sum = warp_sum(sum);
        const float log_sum = logf(sum);
        float h = 0.0f;
        for (int k = lane; k < a.K; k += 32) {
            const float d = (p_of[k] - top) / a.z, p = j_of[k] < 0 ? 0.0f : expf(d) / sum;
            if (p != 0.0f) h += p * (d - log_sum); // NaN goes on
            p_of[k] = p;
        }
        entropy = warp_sum(h);
        if (lane == 0) soft_flag = top != -INFINITY || bad != 0.0f; // some entry has a probability
    } else if (hard || teacher) {
        // the largest logit and the sums
        float base = 0.0f; // what is subtracted: the largest, while there is a finite one
        float2 sum = make_float2(0.0f, 0.0f), sum_soft = sum;
        auto raise = [&](float top) {
            if (top > mine.top) {
                const float d = mine.top - top;
                const float f = fast_exp2(d * l), g = fast_exp2(d * lz);
                sum = make_float2(sum.x * f, sum.y * f);
                if (SUMS) sum_soft = make_float2(sum_soft.x * g, sum_soft.y * g);
                base = mine.top = top;
            }
        };
        auto take = [&](float2 v) {
            float2 e, f;
            exponentials<SUMS>(add2(v, make_float2(-base, -base)), l, lz, &e, &f);
            sum = add2(sum, e);
            if (SUMS) sum_soft = add2(sum_soft, f);
        };
        auto take8 = [&](const uint4& u) {
            const float2 m = unpack16(max16<BF16>(max16<BF16>(u.x, u.y), max16<BF16>(u.z, u.w)), BF16);
            raise(fmaxf(m.x, m.y));
            take(unpack16(u.x, BF16));
            take(unpack16(u.y, BF16));
            take(unpack16(u.z, BF16));
            take(unpack16(u.w, BF16));
        };
        if (VEC) {
            int c = head + self * 8;
            for (; c + (kAtOnce - 1) * everyone * 8 < rest; c += kAtOnce * everyone * 8) {
                uint4 u[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) u[k] = *reinterpret_cast<const uint4*>(s + c + k * everyone * 8);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) take8(u[k]);
            }
            for (; c < rest; c += everyone * 8) take8(*reinterpret_cast<const uint4*>(s + c));
        }
        // what lies before and behind the vectors: fewer than 16 elements where there are any
        for (int c = self < head ? self : rest + self - head; c < a.V; c += everyone * 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = c + j * everyone;
                v[j] = at < a.V && (j == 0 || !VEC) ? load16(s, at, BF16) : -INFINITY;
            }
            float top = v[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = fmaxf(top, v[j]);
            raise(top);
#pragma unroll
            for (int j = 0; j < 8; j += 2) take(make_float2(v[j], v[j + 1]));
            if (VEC) break;
        }
        mine.sum = sum.x + sum.y;
        mine.soft = sum_soft.x + sum_soft.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Tops other;
            other.top = __shfl_xor_sync(0xffffffffu, mine.top, o);
            other.sum = __shfl_xor_sync(0xffffffffu, mine.sum, o);
            other.soft = __shfl_xor_sync(0xffffffffu, mine.soft, o);
            mine = join(mine, other, l, lz);
        }
    }
    if (lane == 0) tops[warp] = mine;
    __syncthreads();
    const bool soft = teacher && soft_flag;

    if (!hard && !soft) { // nothing to learn from this row, whatever it holds
        if (tid == 0) a.loss[row] = 0.0f;
        if (a.grad) {
            for (int c = head + tid * 8; c < rest; c += kLossThreads * 8) *reinterpret_cast<uint4*>(ds + c) = make_uint4(0, 0, 0, 0);
            if (tid < head) ds[tid] = 0;
            for (int c = rest + tid; c < a.V; c += kLossThreads) ds[c] = 0;
        }
        return;
    }
    Tops all = tops[0];
#pragma unroll
    for (int k = 1; k < kLossWarps; ++k) all = join(all, tops[k], l, lz);
    const float sum_hard = all.sum, sum_soft = SUMS ? all.soft : all.sum;
    const float base = all.top == -INFINITY ? 0.0f : all.top;
    // the gradient: f_hard 2^(l1 (s - top)) + f_soft 2^(lz (s - top))
    const float g = w * a.scale, g_soft = g * a.soft * a.z;
    const float f_hard = hard ? g * a.hard / sum_hard : 0.0f, f_soft = soft ? g_soft / sum_soft : 0.0f;
    auto slope = [&](float2 v) {
        float2 e, f;
        exponentials<SUMS>(add2(v, make_float2(-base, -base)), l, lz, &e, &f);
        if (SUMS) return fma2(make_float2(f_hard, f_hard), e, mul2(make_float2(f_soft, f_soft), f));
        return mul2(make_float2(f_hard + f_soft, f_hard + f_soft), e);
    };
    auto slope1 = [&](float v) { return slope(make_float2(v, v)).x; };
    // the gradient's value at an entry: an index that occurs twice has the same, whole value both times.  Each entry
    // looks at all K: nothing beside a row for tens of them, but K^2 steps (16384 rows of 2000: K = 16 57 us, 64 63,
    // 256 334, 1024 3610)
    auto merged = [&](int k) {
        const int j = j_of[k];
        float p = 0.0f;
        for (int i = 0; i < a.K; ++i)
            if (j_of[i] == j) p += p_of[i];
        float v = slope1(s_of[k]) - g_soft * p;
        if (hard && j == target) v -= g * a.hard;
        return v;
    };

    bool listed = false; // the target is among the teacher's
    if (self < 0 || (!teacher && warp == 0)) {
        float cross = 0.0f; // sum p log q'
        if (soft) {
            float h = 0.0f;
            const float log_sum = logf(sum_soft);
            for (int k = lane; k < a.K; k += 32) {
                const float p = p_of[k];
                if (p != 0.0f) h += p * ((s_of[k] - all.top) / a.z - log_sum);
                listed = listed || j_of[k] == target;
            }
            cross = warp_sum(h);
            listed = __any_sync(0xffffffffu, listed);
            if (a.grad && a.K <= kFewTeachers)
                for (int k = lane; k < a.K; k += 32) v_of[k] = merged(k);
        }
        if (lane == 0) {
            float v = 0.0f;
            if (hard) v += a.hard * (logf(sum_hard) - (s_target - all.top));
            if (soft) v += a.soft * a.z * a.z * (entropy - cross);
            a.loss[row] = w * v;
        }
    }
    if (!a.grad) return;
    if (self >= 0) {
        auto write8 = [&](int c, const uint4& u) {
            const float2 v0 = slope(unpack16(u.x, BF16)), v1 = slope(unpack16(u.y, BF16)), v2 = slope(unpack16(u.z, BF16)), v3 = slope(unpack16(u.w, BF16));
            *reinterpret_cast<uint4*>(ds + c) = make_uint4(pack16(v0.x, v0.y, BF16), pack16(v1.x, v1.y, BF16), pack16(v2.x, v2.y, BF16), pack16(v3.x, v3.y, BF16));
        };
        if (VEC) {
            int c = head + self * 8;
            for (; c + (kAtOnce - 1) * everyone * 8 < rest; c += kAtOnce * everyone * 8) {
                uint4 u[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) u[k] = *reinterpret_cast<const uint4*>(s + c + k * everyone * 8);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) write8(c + k * everyone * 8, u[k]);
            }
            for (; c < rest; c += everyone * 8) write8(c, *reinterpret_cast<const uint4*>(s + c));
            if (self < head) store16(ds, self, slope1(load16(s, self, BF16)), BF16);
        }
#pragma unroll 8
        for (int c = rest + self; c < a.V; c += everyone) store16(ds, c, slope1(load16(s, c, BF16)), BF16);
    }
    __syncthreads(); // every element has its sum's part
    if (soft && a.K <= kFewTeachers) {
        if (self < 0)
            for (int k = lane; k < a.K; k += 32)
                if (j_of[k] >= 0) store16(ds, j_of[k], v_of[k], BF16);
    } else if (soft) {
        for (int k = tid; k < a.K; k += kLossThreads)
            if (j_of[k] >= 0) store16(ds, j_of[k], merged(k), BF16);
    }
    if (hard && !listed && tid == 0) store16(ds, target, slope1(s_target) - g * a.hard, BF16);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

using LossKernel = void (*)(LossArgs);

template <int BF16, int VEC, int THREADS> LossKernel pick_loss(int sums)
{
    switch (sums) {
    case 0: return zero_distill_kernel<BF16, VEC, 0, THREADS>;
    case 2: return zero_distill_kernel<BF16, VEC, 2, THREADS>;
    case 4: return zero_distill_kernel<BF16, VEC, 4, THREADS>;
    default: return zero_distill_kernel<BF16, VEC, 1, THREADS>;
    }
}

// Short rows take few threads and many rows an SM: a row's time is then the
// latency of its steps (16384 rows of 1000 logits, 64 of a teacher's: 64 threads
// 58 us, 128 87; of 4000 without a teacher 55, 68, with 20 of a teacher's 102, 84:
// its warp leaves only one for the row; 9133 rows of 10007 with 64: 128 threads
// 88, 256 159).  Long ones 256, four an SM, so that L2 holds all of them for the
// second pass (8192 rows of 44629 with 64: 275 us, 128 threads 390, 512 380; the
// row in shared memory instead, two CTAs an SM, 375).  A row is one CTA's however
// few there are: 1 to 64 rows of 10007 7 us, of 44629 10, of 150000 23 to 34; 509
// of them 9, 24 and 79.  (At 48 registers ten of the forms with 64 or 128 threads
// spill 4 to 8 bytes.)
constexpr int64_t kShortRows = 16384;
int64_t shortest_rows(int64_t K) { return K > 0 ? 2560 : 6144; }

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
    const int sums = !both ? 0 : temperature == 2.0f ? 2 : temperature == 4.0f ? 4 : 1;
    // every row of the gradient starts as far from a boundary of 16 bytes as that of the logits
    const bool vec = !dlogits || ((addr(logits) - addr(dlogits)) % 16 == 0 && (ldl - lddl) % 8 == 0);
    const int bf16 = type == ZERO_TYPE_BF16;
    LossKernel fn;
    const int threads = V < shortest_rows(K) ? 64 : V < kShortRows ? 128 : 256;
    if (threads == 64) fn = bf16 ? (vec ? pick_loss<1, 1, 64>(sums) : pick_loss<1, 0, 64>(sums)) : (vec ? pick_loss<0, 1, 64>(sums) : pick_loss<0, 0, 64>(sums));
    else if (threads == 128) fn = bf16 ? (vec ? pick_loss<1, 1, 128>(sums) : pick_loss<1, 0, 128>(sums)) : (vec ? pick_loss<0, 1, 128>(sums) : pick_loss<0, 0, 128>(sums));
    else fn = bf16 ? (vec ? pick_loss<1, 1, 256>(sums) : pick_loss<1, 0, 256>(sums)) : (vec ? pick_loss<0, 1, 256>(sums) : pick_loss<0, 0, 256>(sums));
    return launch_after(fn, a, T, threads, static_cast<int>(K) * 16, 1, static_cast<cudaStream_t>(cuda_stream));
}
