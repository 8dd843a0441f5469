// Embedding lookup y[t] = scale table[ids[t]] and its gradient
// dtable[v] = scale (sum of dy[t] over the tokens t with ids[t] = v).
//
// The lookup is bound by HBM: a warp copies a piece of a row with all of its
// reads in flight.  Off 16 bytes both directions go by the 16-byte granules of
// the row that is written (its phase: the elements before it in its first
// granule), and the rows that are read are shifted to them.
//
// The gradient sums each row's tokens in the tokens' order, without atomics on
// values, so that a call repeats its bits.  The tokens are sorted by id with a
// stable radix sort (9 bits a pass: two passes up to 2^18 ids; a block ranks
// its tokens by the lanes' matching digits and finds its place from the blocks'
// digit counts): up to 65536 tokens by one cluster of eight CTAs, which
// exchange counts and tokens through distributed shared memory while the other
// SMs clear the first rows of the table, more by two launches per pass.  Then
// warps walk over the sorted tokens, a chunk of them and a stripe of 256
// columns each, adding rows of dy in registers; a run of equal ids that lies in
// one chunk is written at once, the parts of a longer one go to the workspace
// in fp32 and are added in order by a last launch.  However often an id occurs,
// no warp has more than a chunk of rows to read.
// 16384 tokens, a table of 44629 x 2048 (250 MB, 183 of them written) 60 us: sort
// and cleared rows 12, sums and the other rows without a token 38 (210 MB, 5500
// GB/s), joins 10.  The sort and the joins are latency with HBM nearly idle: a
// fill of the table alone takes 31 (6000 GB/s, by vectors or by bulk copies from
// cleared shared memory alike).
#include "layers.cuh"

namespace {

struct LookArgs {
    const int32_t* ids;
    const void* table;
    void* y;
    long long ldt, ldy, T, items;
    int D, V, pieces;
    float scale;
};

constexpr int kLookPiece = 1024; // columns of a warp's item: four vectors of 8 a lane

// One warp per piece of a token's row.  VEC: rows lie on 16 bytes.  16384 tokens
// of 2048 bf16 elements (91 MB) 15.7 us, 5800 GB/s; off 16 bytes 29 us.
template <int BF16, int VEC> __global__ void __launch_bounds__(256) zero_embed_kernel(const __grid_constant__ LookArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    let_successor_start();
    wait_for_predecessor();
    if (item >= a.items) return;
    const long long t = item / a.pieces;
    const int c0 = static_cast<int>(item - t * a.pieces) * kLookPiece;
    const int id = a.ids[t];
    const bool there = id >= 0 && id < a.V;
    const uint16_t* from = static_cast<const uint16_t*>(a.table) + (there ? id * a.ldt : 0);
    uint16_t* to = static_cast<uint16_t*>(a.y) + t * a.ldy;
    const int phase = VEC ? 0 : phase_of(to);
    uint4 u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = c0 + (k * 32 + lane) * 8 - phase;
        u[k] = make_uint4(0, 0, 0, 0);
        if (there && c < a.D) u[k] = VEC ? *reinterpret_cast<const uint4*>(from + c) : load_any(from, c, a.D);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c = c0 + (k * 32 + lane) * 8 - phase;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        add8(v, u[k], BF16);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = there ? v[j] * a.scale : 0.0f;
        if (!VEC) put_granule(to, c, a.D, pack8(v, BF16));
        else if (c < a.D) *reinterpret_cast<uint4*>(to + c) = pack8(v, BF16);
    }
}

// ---------------------------------------------------------------------------
// Stable radix sort of (id, token)
// ---------------------------------------------------------------------------

constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSortThreads = kDigits, kSortWarps = kSortThreads / 32; // a thread per digit
constexpr int kRounds = 8, kSortTokens = kRounds * kSortThreads;       // tokens of a block

struct SortArgs {
    const int32_t* ids;  // the first pass: the ids in order
    const int2* from;    // later ones: (id, token)
    int2* to;
    uint32_t* counts;    // [blocks + 1][kDigits] of this pass: each block's tokens with a digit, then sums of them
    uint32_t* next;      // the same of the next pass, null in the last
    long long T;
    int V, shift, blocks, all_counts;
};

// An id that names no row sorts behind every other one.
__device__ __forceinline__ int sort_key(int id, int V) { return id >= 0 && id < V ? id : V; }

// Digit counts of each block for the first pass; the later passes' counts
// become 0 (the passes before them add to these).
__global__ void __launch_bounds__(kSortThreads) zero_sort_count_kernel(const __grid_constant__ SortArgs a)
{
    __shared__ uint32_t count[kDigits];
    let_successor_start();
    count[threadIdx.x] = 0;
    __syncthreads();
    wait_for_predecessor();
    const long long t0 = static_cast<long long>(blockIdx.x) * kSortTokens;
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const long long t = t0 + k * kSortThreads + threadIdx.x;
        if (t < a.T) atomicAdd(&count[sort_key(a.ids[t], a.V) & (kDigits - 1)], 1u);
    }
    __syncthreads();
    a.counts[static_cast<long long>(blockIdx.x) * kDigits + threadIdx.x] = count[threadIdx.x];
    for (int p = 1; p < a.all_counts; ++p)
        a.counts[(static_cast<long long>(p) * (a.blocks + 1) + blockIdx.x) * kDigits + threadIdx.x] = 0;
}

// A warp per digit: its tokens in each block become those in the blocks before
// it, and behind the last block stands the sum of all.
__global__ void __launch_bounds__(256) zero_sort_scan_kernel(const __grid_constant__ SortArgs a)
{
    const int lane = threadIdx.x & 31, d = static_cast<int>(blockIdx.x) * 8 + static_cast<int>(threadIdx.x >> 5);
    let_successor_start();
    wait_for_predecessor();
    uint32_t before = 0;
    for (long long b0 = 0; b0 < a.blocks; b0 += 32) {
        uint32_t* p = a.counts + (b0 + lane) * kDigits + d;
        const uint32_t own = b0 + lane < a.blocks ? *p : 0;
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
        if (b0 + lane < a.blocks) *p = before + sum - own;
        before += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) a.counts[static_cast<long long>(a.blocks) * kDigits + d] = before;
}

// One pass: each token's place is the start of its digit, the tokens with the
// digit in earlier blocks, those in earlier warps of the block, and those
// earlier in the warp.
__global__ void __launch_bounds__(kSortThreads) zero_sort_pass_kernel(const __grid_constant__ SortArgs a)
{
    __shared__ uint32_t count[kSortWarps][kDigits];
    __shared__ uint32_t warp_total[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = threadIdx.x;
    let_successor_start();
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) count[k][d] = 0;
    __syncthreads();
    wait_for_predecessor();
    const long long t0 = static_cast<long long>(blockIdx.x) * kSortTokens + warp * (kRounds * 32);
    int key[kRounds], token[kRounds];
    uint32_t rank[kRounds];
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const long long t = t0 + k * 32 + lane;
        key[k] = token[k] = 0;
        if (t < a.T) {
            if (a.ids) {
                key[k] = sort_key(a.ids[t], a.V);
                token[k] = static_cast<int>(t);
            } else {
                const int2 p = a.from[t];
                key[k] = p.x;
                token[k] = p.y;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        const bool live = t0 + k * 32 + lane < a.T;
        const int digit = live ? (key[k] >> a.shift) & (kDigits - 1) : kDigits;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        const uint32_t before = live ? count[warp][digit] : 0;
        rank[k] = before + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (live && (same >> lane) == 1) count[warp][digit] = before + __popc(same); // the last of them
        __syncwarp();
    }
    // tokens with digit d in earlier blocks and in all
    const uint32_t earlier = a.counts[static_cast<long long>(blockIdx.x) * kDigits + d], all = a.counts[static_cast<long long>(a.blocks) * kDigits + d];
    // the start of digit d: an exclusive sum over the digits
    uint32_t sum = all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t n = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += n;
    }
    if (lane == 31) warp_total[warp] = sum;
    __syncthreads();
    uint32_t at = earlier + sum - all;
    for (int k = 0; k < warp; ++k) at += warp_total[k];
#pragma unroll
    for (int k = 0; k < kSortWarps; ++k) {
        const uint32_t n = count[k][d];
        count[k][d] = at;
        at += n;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRounds; ++k) {
        if (t0 + k * 32 + lane >= a.T) continue;
        const uint32_t to = count[warp][(key[k] >> a.shift) & (kDigits - 1)] + rank[k];
        a.to[to] = make_int2(key[k], token[k]);
        if (a.next) atomicAdd(&a.next[static_cast<long long>(to / kSortTokens) * kDigits + ((key[k] >> (a.shift + kDigitBits)) & (kDigits - 1))], 1u);
    }
}

// Zeros to a row, by a warp.
template <int VEC> __device__ __forceinline__ void clear_row(uint16_t* row, int D, int lane)
{
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int c = lane * 8 - (VEC ? 0 : phase_of(row)); c < D; c += 256) {
        if (!VEC) put_granule(row, c, D, zero);
        else *reinterpret_cast<uint4*>(row + c) = zero;
    }
}

// The whole sort by one cluster: a CTA holds every eighth part of the order in
// its shared memory, a thread ROUNDS tokens in registers.  Per pass the CTAs
// rank their tokens, read each other's digit counts, and write the tokens to
// their places in each other's memory.  The clusters behind the first one
// write zeros to the table's first `clear` rows meanwhile.
constexpr int kCluster = 8, kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32;

template <int ROUNDS> constexpr int kClusterSortSmem = ROUNDS * kClusterThreads * 8 + kClusterWarps * kDigits * 2 + 2 * kDigits * 4;

struct ClusterSortArgs {
    const int32_t* ids;
    int2* to;
    uint16_t* dtable;
    long long lddt, clear;
    int T, V, D, passes, vec;
};

__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t at_peer(const void* p, uint32_t rank)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
    return at;
}

template <int ROUNDS> __global__ void __launch_bounds__(kClusterThreads) zero_sort_cluster_kernel(const __grid_constant__ ClusterSortArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    constexpr int kTokens = ROUNDS * kClusterThreads;
    int2* pairs = reinterpret_cast<int2*>(raw);                                  // [kTokens]
    uint16_t* count = reinterpret_cast<uint16_t*>(raw + kTokens * 8);            // [kClusterWarps][kDigits]
    uint32_t* total = reinterpret_cast<uint32_t*>(count + kClusterWarps * kDigits); // [kDigits], read by the peers
    uint32_t* base = total + kDigits;                                            // [kDigits]
    __shared__ uint32_t warp_total[kDigits / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    let_successor_start();
    wait_for_predecessor();
    if (blockIdx.x >= kCluster) {
        const int warps = (gridDim.x - kCluster) * kClusterWarps;
        for (long long v = (blockIdx.x - kCluster) * kClusterWarps + warp; v < a.clear; v += warps) {
            uint16_t* row = a.dtable + v * a.lddt;
            if (a.vec) clear_row<1>(row, a.D, lane);
            else clear_row<0>(row, a.D, lane);
        }
        return;
    }
    const int rank = static_cast<int>(blockIdx.x), t0 = rank * kTokens + warp * (ROUNDS * 32);
    int key[ROUNDS], token[ROUNDS];
    uint32_t place[ROUNDS];
#pragma unroll
    for (int k = 0; k < ROUNDS; ++k) {
        token[k] = t0 + k * 32 + lane;
        key[k] = token[k] < a.T ? sort_key(a.ids[token[k]], a.V) : 0;
    }
    for (int pass = 0, shift = 0; pass < a.passes; ++pass, shift += kDigitBits) {
        for (int i = tid; i < kClusterWarps * kDigits / 2; i += kClusterThreads) reinterpret_cast<uint32_t*>(count)[i] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const bool live = t0 + k * 32 + lane < a.T;
            const int digit = live ? (key[k] >> shift) & (kDigits - 1) : kDigits;
            const uint32_t same = __match_any_sync(0xffffffffu, digit);
            const uint32_t before = live ? count[warp * kDigits + digit] : 0;
            place[k] = before + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (live && (same >> lane) == 1) count[warp * kDigits + digit] = static_cast<uint16_t>(before + __popc(same)); // the last of them
            __syncwarp();
        }
        __syncthreads();
        if (tid < kDigits) { // tokens with this digit in the warps before each one
            uint32_t n = 0;
#pragma unroll
            for (int w = 0; w < kClusterWarps; ++w) {
                const uint32_t own = count[w * kDigits + tid];
                count[w * kDigits + tid] = static_cast<uint16_t>(n);
                n += own;
            }
            total[tid] = n;
        }
        cluster_barrier(); // the counts are there, and every CTA has its tokens in registers
        uint32_t all = 0, earlier = 0, sum = 0;
        if (tid < kDigits) {
#pragma unroll
            for (int r = 0; r < kCluster; ++r) {
                uint32_t n;
                asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(n) : "r"(at_peer(total + tid, r)) : "memory");
                all += n;
                if (r < rank) earlier += n;
            }
            sum = all;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t n = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += n;
            }
            if (lane == 31) warp_total[warp] = sum;
        }
        __syncthreads();
        if (tid < kDigits) {
            uint32_t at = earlier + sum - all;
            for (int w = 0; w < warp; ++w) at += warp_total[w];
            base[tid] = at;
        }
        __syncthreads();
        const bool last = pass + 1 == a.passes;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            if (t0 + k * 32 + lane >= a.T) continue;
            const int digit = (key[k] >> shift) & (kDigits - 1);
            const uint32_t to = base[digit] + count[warp * kDigits + digit] + place[k];
            if (last) {
                a.to[to] = make_int2(key[k], token[k]);
            } else {
                asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(at_peer(pairs + to % kTokens, to / kTokens)), "r"(key[k]), "r"(token[k])
                             : "memory");
            }
        }
        cluster_barrier(); // the tokens have arrived, and no CTA reads another one's counts any more
        if (last) break;
#pragma unroll
        for (int k = 0; k < ROUNDS; ++k) {
            const int at = warp * (ROUNDS * 32) + k * 32 + lane;
            if (rank * kTokens + at < a.T) key[k] = pairs[at].x, token[k] = pairs[at].y;
        }
    }
}

// ---------------------------------------------------------------------------
// Sums over runs of equal ids
// ---------------------------------------------------------------------------

constexpr int kStripe = 256;   // columns of a warp: 8 a lane
constexpr int kZeroRows = 8;   // rows of the table that a warp looks up and clears where they have no token

struct RunArgs {
    const int2* sorted;
    const void* dy;
    void* dtable;
    float* parts;        // [chunks][2][pitch], by granules of the row: of the run that began before the chunk, of the one that goes on behind it
    long long lddy, lddt, T, sum_tasks, join_tasks, tasks, cleared; // rows of the table below `cleared` are 0 already
    int D, V, stripes, chunk, add, pitch;
    float scale;
};

// Eight elements of a row from column c on.
template <int VEC> __device__ __forceinline__ uint4 get_row(const uint16_t* row, int c, int D)
{
    if constexpr (!VEC) return load_any(row, c, D);
    return c < D ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
}

// A run's sum, plus what the table's gradient held (zeros where it does not
// count), to its row.
template <int BF16, int VEC>
__device__ __forceinline__ void put_row(const RunArgs& a, uint16_t* row, int c, const float (&sum)[8], const uint4& old)
{
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = sum[j] * a.scale;
    if (a.add) add8(v, old, BF16);
    if constexpr (!VEC) put_granule(row, c, a.D, pack8(v, BF16));
    else if (c < a.D) *reinterpret_cast<uint4*>(row + c) = pack8(v, BF16);
}

// Rows of the table without a token become 0: each lane looks its row up among
// the sorted ids.
template <int VEC> __device__ __forceinline__ void clear_rows(const RunArgs& a, long long v0, int lane)
{
    const int v = static_cast<int>(v0) + lane;
    bool absent = lane < kZeroRows && v < a.V;
    if (absent) {
        long long lo = 0, hi = a.T; // first place whose id is v or above
        while (lo < hi) {
            const long long mid = (lo + hi) >> 1;
            if (a.sorted[mid].x < v) lo = mid + 1;
            else hi = mid;
        }
        absent = lo >= a.T || a.sorted[lo].x != v;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, absent);
    while (todo) {
        const int k = __ffs(todo) - 1;
        todo &= todo - 1;
        uint16_t* row = static_cast<uint16_t*>(a.dtable) + (v0 + k) * a.lddt;
        clear_row<VEC>(row, a.D, lane);
    }
}

// CTAs an SM: about as many as the rows in flight leave registers for (aligned
// rows that are written spill 24 bytes at three, unaligned ones that are added to
// 108 at four).
template <int BF16, int VEC, int ADD> __global__ void __launch_bounds__(256, VEC ? (ADD ? 2 : 3) : 4) zero_embed_grad_kernel(const __grid_constant__ RunArgs a)
{
    constexpr int kAhead = VEC ? 8 : 4; // rows in flight (two granules each off 16 bytes)
    const int lane = threadIdx.x & 31;
    const long long task = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    let_successor_start();
    wait_for_predecessor();
    if (task >= a.tasks) return;
    if (task >= a.sum_tasks) {
        clear_rows<VEC>(a, a.cleared + (task - a.sum_tasks) * kZeroRows, lane);
        return;
    }
    const long long chunk = task / a.stripes, first = chunk * a.chunk, end = min(a.T, first + a.chunk);
    const int col = static_cast<int>(task - chunk * a.stripes) * kStripe + lane * 8;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
    float sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
    bool begun = first > 0 && a.sorted[first - 1].x == a.sorted[first].x; // the run began before the chunk
    bool open = false;                                                     // the sum holds a row
    auto put_part = [&]() {
        if (col >= a.pitch) return;
        float4* part = reinterpret_cast<float4*>(a.parts + (chunk * 2 + (begun ? 0 : 1)) * a.pitch + col);
        part[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
        part[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
    };
    for (long long s = first; s < end; s += 32) {
        const int2 none = make_int2(a.V, 0);
        const int2 mine = s + lane < end ? a.sorted[s + lane] : none;
        // which tokens are there, and which end their run: one bit each, so that the sums below shuffle nothing
        const int next = s + lane + 1 < a.T ? a.sorted[s + lane + 1].x : a.V;
        const int n = __popc(__ballot_sync(0xffffffffu, mine.x < a.V));
        const uint32_t ends = __ballot_sync(0xffffffffu, mine.x != next);
        for (int i0 = 0; i0 < n; i0 += kAhead) {
            uint4 u[kAhead], o[ADD ? kAhead : 1] = {};
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const uint16_t* row = dy + __shfl_sync(0xffffffffu, mine.y, i0 + i) * a.lddy;
                u[i] = make_uint4(0, 0, 0, 0);
                o[ADD ? i : 0] = make_uint4(0, 0, 0, 0);
                if (VEC && !ADD) {
                    if (i0 + i < n) u[i] = get_row<VEC>(row, col, a.D);
                    continue;
                }
                const uint16_t* to = static_cast<const uint16_t*>(a.dtable) + __shfl_sync(0xffffffffu, mine.x, i0 + i) * a.lddt;
                const int c = VEC ? col : col - phase_of(to);
                if (i0 + i < n) {
                    u[i] = get_row<VEC>(row, c, a.D);
                    // the table's row as it was: read with the others, for the token that ends its run
                    if (ADD && (ends >> (i0 + i) & 1)) o[ADD ? i : 0] = get_row<VEC>(to, c, a.D);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (i0 + i >= n) break;
                add8(sum, u[i], BF16);
                open = true;
                if (!(ends >> (i0 + i) & 1)) continue;
                uint16_t* to = static_cast<uint16_t*>(a.dtable) + __shfl_sync(0xffffffffu, mine.x, i0 + i) * a.lddt;
                if (begun) put_part();
                else put_row<BF16, VEC>(a, to, VEC ? col : col - phase_of(to), sum, o[ADD ? i : 0]);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[j] = 0.0f;
                begun = open = false;
            }
        }
        if (n < 32) break; // behind the last id, or at the chunk's end
    }
    if (open) put_part(); // the run goes on behind the chunk
}

// The same place of eight parts (the first n; later ones are not read): one
// statement, since the compiler adds each part before it reads the next
// otherwise (16384 tokens, 2048 columns, runs of up to 33 parts: 20 us).
__device__ __forceinline__ void read_eight(const float* from, long long pitch, int n, float (&v)[8][4])
{
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0.0f;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.gt.s32 p, %40, 0;\n\t@p ld.global.v4.f32 {%0, %1, %2, %3}, [%32];\n\t"
                 "setp.gt.s32 p, %40, 1;\n\t@p ld.global.v4.f32 {%4, %5, %6, %7}, [%33];\n\t"
                 "setp.gt.s32 p, %40, 2;\n\t@p ld.global.v4.f32 {%8, %9, %10, %11}, [%34];\n\t"
                 "setp.gt.s32 p, %40, 3;\n\t@p ld.global.v4.f32 {%12, %13, %14, %15}, [%35];\n\t"
                 "setp.gt.s32 p, %40, 4;\n\t@p ld.global.v4.f32 {%16, %17, %18, %19}, [%36];\n\t"
                 "setp.gt.s32 p, %40, 5;\n\t@p ld.global.v4.f32 {%20, %21, %22, %23}, [%37];\n\t"
                 "setp.gt.s32 p, %40, 6;\n\t@p ld.global.v4.f32 {%24, %25, %26, %27}, [%38];\n\t"
                 "setp.gt.s32 p, %40, 7;\n\t@p ld.global.v4.f32 {%28, %29, %30, %31}, [%39];\n\t}"
                 : "+f"(v[0][0]), "+f"(v[0][1]), "+f"(v[0][2]), "+f"(v[0][3]), "+f"(v[1][0]), "+f"(v[1][1]), "+f"(v[1][2]), "+f"(v[1][3]),
                   "+f"(v[2][0]), "+f"(v[2][1]), "+f"(v[2][2]), "+f"(v[2][3]), "+f"(v[3][0]), "+f"(v[3][1]), "+f"(v[3][2]), "+f"(v[3][3]),
                   "+f"(v[4][0]), "+f"(v[4][1]), "+f"(v[4][2]), "+f"(v[4][3]), "+f"(v[5][0]), "+f"(v[5][1]), "+f"(v[5][2]), "+f"(v[5][3]),
                   "+f"(v[6][0]), "+f"(v[6][1]), "+f"(v[6][2]), "+f"(v[6][3]), "+f"(v[7][0]), "+f"(v[7][1]), "+f"(v[7][2]), "+f"(v[7][3])
                 : "l"(from), "l"(from + pitch), "l"(from + 2 * pitch), "l"(from + 3 * pitch), "l"(from + 4 * pitch), "l"(from + 5 * pitch),
                   "l"(from + 6 * pitch), "l"(from + 7 * pitch), "r"(n)
                 : "memory");
}

// The parts of a run that passes a chunk's end, added in order by a warp of
// the chunk that it begins in: four columns a lane, sixteen parts in flight.
// Bound by latency.
constexpr int kJoinStripe = 128, kJoinAhead = 16;

template <int BF16, int VEC> __global__ void __launch_bounds__(128) zero_embed_join_kernel(const __grid_constant__ RunArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long task = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    let_successor_start();
    wait_for_predecessor();
    if (task >= a.join_tasks) return;
    const int stripes = (a.pitch + kJoinStripe - 1) / kJoinStripe;
    const long long chunk = task / stripes, first = chunk * a.chunk, end = first + a.chunk;
    if (end >= a.T) return;
    const int key = a.sorted[end - 1].x, next = a.sorted[end].x, previous = first > 0 ? a.sorted[first - 1].x : -1;
    if (key >= a.V || next != key || previous == key) return;
    // the chunks behind this one that begin with the run
    const long long chunks = (a.T + a.chunk - 1) / a.chunk;
    long long last = chunk; // the last chunk that holds a part
    while (true) {
        const long long c = last + 1 + lane;
        const bool in = c < chunks && a.sorted[c * a.chunk].x == key;
        const uint32_t all = __ballot_sync(0xffffffffu, in);
        const int n = all == 0xffffffffu ? 32 : __ffs(~all) - 1;
        last += n;
        if (n < 32) break;
    }
    const int c0 = static_cast<int>(task - chunk * stripes) * kJoinStripe;
    const int at = min(c0 + lane * 4, a.pitch - 4); // lanes behind the parts read their end, and write nothing
    uint16_t* row = static_cast<uint16_t*>(a.dtable) + key * a.lddt;
    const int col = VEC ? at : at - phase_of(row);
    float sum[4], old[4];
    const float4 tail = *reinterpret_cast<const float4*>(a.parts + (chunk * 2 + 1) * a.pitch + at);
    sum[0] = tail.x, sum[1] = tail.y, sum[2] = tail.z, sum[3] = tail.w;
#pragma unroll
    for (int j = 0; j < 4; ++j) old[j] = a.add && col + j >= 0 && col + j < a.D ? load16(row, col + j, BF16) : 0.0f;
    for (long long c = chunk + 1; c <= last; c += kJoinAhead) {
        const int n = static_cast<int>(min(static_cast<long long>(kJoinAhead), last + 1 - c));
        float v[kJoinAhead / 8][8][4];
#pragma unroll
        for (int h = 0; h < kJoinAhead / 8; ++h) read_eight(a.parts + (c + 8 * h) * 2 * a.pitch + at, 2ll * a.pitch, n - 8 * h, v[h]);
#pragma unroll
        for (int k = 0; k < kJoinAhead; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] += v[k / 8][k % 8][j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = sum[j] * a.scale + old[j];
    if (c0 + lane * 4 >= a.pitch) return;
    if (VEC) {
        *reinterpret_cast<uint2*>(row + at) = make_uint2(pack16(sum[0], sum[1], BF16), pack16(sum[2], sum[3], BF16));
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (col + j >= 0 && col + j < a.D) store16(row, col + j, sum[j], BF16);
    }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

constexpr int64_t kMostIds = int64_t{1} << 30;

bool bad_embed(int64_t T, int64_t D, int64_t V, float scale, int32_t type)
{
    return T < 0 || T > kMostExtent || D < 1 || D > kMostIds || V < 1 || V > kMostIds || std::max(T, V) * D > kMostElements ||
           !(scale > -INFINITY && scale < INFINITY) || (type != ZERO_TYPE_FP16 && type != ZERO_TYPE_BF16);
}

// The layout of a gradient's workspace and the sizes of its launches.
struct GradPlan {
    int cluster;         // rounds of the sort by one cluster, 0: a launch per pass
    int blocks, passes, chunk;
    int64_t chunks, stripes, pitch;
    int2* pairs[2];
    uint32_t* counts;
    float* parts;
    int64_t bytes;
};

GradPlan plan_grad(int64_t T, int64_t D, int64_t V, void* workspace)
{
    GradPlan p{};
    for (int r = 1; r <= 8 && !p.cluster; r *= 2)
        if (T <= r * kCluster * kClusterThreads) p.cluster = r;
    p.blocks = p.cluster ? 0 : static_cast<int>((T + kSortTokens - 1) / kSortTokens);
    int bits = 1;
    while ((V >> bits) != 0) ++bits; // of V itself, which stands for no row
    p.passes = (bits + kDigitBits - 1) / kDigitBits;
    p.pitch = up(D + 7, 8); // granules of a row that starts anywhere
    p.stripes = (p.pitch + kStripe - 1) / kStripe;
    // short chunks where there are few: a chunk's rows follow on each other (up to 16 warps an SM: 2432 chunks and
    // stripes on 152); longer ones once there are warps enough, so that fewer runs are cut (8192 of them from 32 tokens
    // a chunk on).  Chunks of 4, 8, 16, 32, 64, 128 and 256 tokens, us, with the gradient added to bf16 rows (fp16 for
    // 331 columns): 1009 tokens x 331 17, 20, 27, 40, 68, 124, 223 (the rule takes 4); 2048 x 2048 21, 16, 18, 21, 29,
    // 46, 78 (8); 16384 x 2048 106, 71, 56, 47, 46, 58, 94 (32); 200000 x 1024 885, 506, 321, 233, 190, 173, 189 (96:
    // 178); 1e6 x 64 3066, 1556, 880, 520, 347, 269, 219 (96: 294)
    p.chunk = 4;
    while (p.chunk < 32 && T * p.stripes > 2432 * p.chunk) p.chunk *= 2;
    if (p.chunk == 32) p.chunk = static_cast<int>(std::min<int64_t>(256, std::max<int64_t>(32, T * p.stripes / 8192 / 32 * 32)));
    p.chunks = (T + p.chunk - 1) / p.chunk;
    Carver c{static_cast<unsigned char*>(workspace)};
    p.pairs[0] = static_cast<int2*>(c.take(T * 8));
    p.pairs[1] = p.cluster ? p.pairs[0] : static_cast<int2*>(c.take(T * 8));
    p.counts = static_cast<uint32_t*>(c.take(p.cluster ? 0 : static_cast<int64_t>(p.passes) * (p.blocks + 1) * kDigits * 4));
    p.parts = static_cast<float*>(c.take(p.chunks * 2 * p.pitch * 4));
    p.bytes = c.used;
    return p;
}

// Of the table's gradient, cleared during a sort by one cluster, and the CTAs that
// do it (with the sort's eight 18 clusters, one CTA an SM).  44629 x 2048 with 1024,
// 16384 and 65536 tokens: nothing cleared ahead 45, 66 and 132 us; 20 MB 42, 64,
// 132; 40 MB 43, 62, 132; 80 MB 48, 66, 130.  64 CTAs 46, 62, 132; 144 as 136.
constexpr int64_t kClearBytes = 40 << 20;
constexpr int kClearCtas = 136;

using ClusterSort = void (*)(ClusterSortArgs);

template <int ROUNDS> int sort_by_cluster(const ClusterSortArgs& a, cudaStream_t stream)
{
    const int rc = allow_smem(reinterpret_cast<const void*>(static_cast<ClusterSort>(zero_sort_cluster_kernel<ROUNDS>)), kClusterSortSmem<ROUNDS>);
    if (rc) return rc;
    return launch_after(static_cast<ClusterSort>(zero_sort_cluster_kernel<ROUNDS>), a, a.clear ? kCluster + kClearCtas : kCluster, kClusterThreads,
                        kClusterSortSmem<ROUNDS>, kCluster, stream);
}

template <class Kernel> Kernel pick(int bf16, int vec, Kernel k00, Kernel k01, Kernel k10, Kernel k11)
{
    return bf16 ? (vec ? k11 : k10) : (vec ? k01 : k00);
}

// A launch for the first counts, then two per pass (the blocks' sums, the
// tokens' places); ends in pairs[(passes - 1) & 1].
int sort_by_passes(const GradPlan& p, const int32_t* ids, int64_t T, int64_t V, cudaStream_t st)
{
    SortArgs s{};
    s.ids = ids, s.counts = p.counts, s.T = T, s.V = static_cast<int>(V), s.blocks = p.blocks, s.all_counts = p.passes;
    int rc = launch_after(zero_sort_count_kernel, s, p.blocks, kSortThreads, 0, 1, st);
    for (int k = 0; k < p.passes && !rc; ++k) {
        const int64_t each = static_cast<int64_t>(p.blocks + 1) * kDigits;
        s.ids = k == 0 ? ids : nullptr;
        s.from = p.pairs[(k + 1) & 1], s.to = p.pairs[k & 1];
        s.counts = p.counts + k * each, s.next = k + 1 < p.passes ? p.counts + (k + 1) * each : nullptr;
        s.shift = k * kDigitBits;
        if (!(rc = launch_after(zero_sort_scan_kernel, s, kDigits / 8, 256, 0, 1, st)))
            rc = launch_after(zero_sort_pass_kernel, s, p.blocks, kSortThreads, 0, 1, st);
    }
    return rc;
}

} // namespace

extern "C" int zero_embed_forward(const int32_t* ids, const void* table, int64_t ldt, void* y, int64_t ldy, int64_t T, int64_t D,
                                  int64_t V, float scale, int32_t type, void* cuda_stream)
{
    if (bad_embed(T, D, V, scale, type)) return ZERO_EINVAL;
    if (T == 0) return ZERO_OK;
    if (!ids || !table || !y || bad_ld(ldt, D) || bad_ld(ldy, D)) return ZERO_EINVAL;
    if (addr(ids) % 4 || addr(table) % 2 || addr(y) % 2) return ZERO_EALIGN;
    if (share(y, ldy, T, D, table, ldt, V, D) || share(y, ldy, T, D, ids, 2 * T, 1, 2 * T)) return ZERO_EOVERLAP;
    LookArgs a{};
    a.ids = ids, a.table = table, a.y = y, a.ldt = ldt, a.ldy = ldy, a.T = T, a.D = static_cast<int>(D), a.V = static_cast<int>(V);
    const bool vec = D % 8 == 0 && aligned16(table, ldt) && aligned16(y, ldy);
    a.pieces = static_cast<int>((D + (vec ? 0 : 7) + kLookPiece - 1) / kLookPiece);
    a.items = T * a.pieces;
    a.scale = scale;
    if ((a.items + 7) / 8 > INT32_MAX) return ZERO_EINVAL;
    auto fn = pick(type == ZERO_TYPE_BF16, vec, zero_embed_kernel<0, 0>, zero_embed_kernel<0, 1>, zero_embed_kernel<1, 0>, zero_embed_kernel<1, 1>);
    return launch_after(fn, a, (a.items + 7) / 8, 256, 0, 1, static_cast<cudaStream_t>(cuda_stream));
}

extern "C" int zero_embed_workspace(int64_t T, int64_t D, int64_t V, int64_t* bytes)
{
    if (!bytes || bad_embed(T, D, V, 1.0f, ZERO_TYPE_FP16)) return ZERO_EINVAL;
    *bytes = T == 0 ? 0 : plan_grad(T, D, V, nullptr).bytes;
    return ZERO_OK;
}

extern "C" int zero_embed_backward(const int32_t* ids, const void* dy, int64_t lddy, void* dtable, int64_t lddt, int64_t T, int64_t D,
                                   int64_t V, float scale, int32_t add, int32_t type, void* workspace, int64_t workspace_bytes,
                                   void* cuda_stream)
{
    if (bad_embed(T, D, V, scale, type) || !dtable || bad_ld(lddt, D)) return ZERO_EINVAL;
    if (T > 0 && (!ids || !dy || bad_ld(lddy, D))) return ZERO_EINVAL;
    if (addr(dtable) % 2 || (T > 0 && (addr(ids) % 4 || addr(dy) % 2))) return ZERO_EALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
    if (T == 0) {
        if (add) return ZERO_OK;
        return record(cudaMemset2DAsync(dtable, static_cast<size_t>(lddt) * 2, 0, static_cast<size_t>(D) * 2, static_cast<size_t>(V), st));
    }
    if (share(dtable, lddt, V, D, dy, lddy, T, D) || share(dtable, lddt, V, D, ids, 2 * T, 1, 2 * T)) return ZERO_EOVERLAP;
    const GradPlan p = plan_grad(T, D, V, workspace);
    if (!workspace || workspace_bytes < p.bytes) return ZERO_EINVAL;
    if (addr(workspace) % 16) return ZERO_EALIGN;
    if (in_workspace(workspace, p.bytes, dy, lddy, T, D) || in_workspace(workspace, p.bytes, dtable, lddt, V, D) ||
        in_workspace(workspace, p.bytes, ids, 2 * T, 1, 2 * T))
        return ZERO_EOVERLAP;
    const int bf16 = type == ZERO_TYPE_BF16;
    const bool vec = D % 8 == 0 && aligned16(dy, lddy) && aligned16(dtable, lddt);
    RunArgs r{};
    r.dy = dy, r.dtable = dtable, r.parts = p.parts, r.lddy = lddy, r.lddt = lddt, r.T = T, r.D = static_cast<int>(D), r.V = static_cast<int>(V);
    r.pitch = static_cast<int>(vec ? D : p.pitch), r.stripes = (r.pitch + kStripe - 1) / kStripe, r.chunk = p.chunk, r.add = add != 0, r.scale = scale;
    r.sum_tasks = p.chunks * r.stripes;
    r.join_tasks = p.chunks * ((r.pitch + kJoinStripe - 1) / kJoinStripe);
    if (!add && p.cluster) r.cleared = std::min<int64_t>(V, kClearBytes / (2 * D));
    r.tasks = r.sum_tasks + (add ? 0 : (V - r.cleared + kZeroRows - 1) / kZeroRows);
    if ((r.tasks + 7) / 8 > INT32_MAX || (r.join_tasks + 3) / 4 > INT32_MAX) return ZERO_EINVAL;
    int rc = ZERO_OK;
    if (p.cluster) {
        ClusterSortArgs s{};
        s.ids = ids, s.to = p.pairs[0], s.dtable = static_cast<uint16_t*>(dtable), s.lddt = lddt, s.clear = r.cleared;
        s.T = static_cast<int>(T), s.V = static_cast<int>(V), s.D = static_cast<int>(D), s.passes = p.passes, s.vec = vec;
        rc = p.cluster == 1   ? sort_by_cluster<1>(s, st)
             : p.cluster == 2 ? sort_by_cluster<2>(s, st)
             : p.cluster == 4 ? sort_by_cluster<4>(s, st)
                              : sort_by_cluster<8>(s, st);
    } else {
        rc = sort_by_passes(p, ids, T, V, st);
    }
    if (rc) return rc;

    r.sorted = p.pairs[(p.passes - 1) & 1];
    auto sum = add ? pick(bf16, vec, zero_embed_grad_kernel<0, 0, 1>, zero_embed_grad_kernel<0, 1, 1>, zero_embed_grad_kernel<1, 0, 1>, zero_embed_grad_kernel<1, 1, 1>)
                   : pick(bf16, vec, zero_embed_grad_kernel<0, 0, 0>, zero_embed_grad_kernel<0, 1, 0>, zero_embed_grad_kernel<1, 0, 0>, zero_embed_grad_kernel<1, 1, 0>);
    if ((rc = launch_after(sum, r, (r.tasks + 7) / 8, 256, 0, 1, st))) return rc;
    auto join = pick(bf16, vec, zero_embed_join_kernel<0, 0>, zero_embed_join_kernel<0, 1>, zero_embed_join_kernel<1, 0>, zero_embed_join_kernel<1, 1>);
    return launch_after(join, r, (r.join_tasks + 3) / 4, 128, 0, 1, st);
}
