// tables.cu -- block tables and slot maps of the resident pages
// (include/hisparse_pages.h, hisparse_page_tables).
//
// The mathematics.  With need = ceil(len / bs), request r gives back f_r =
// max(held - max(need, shared), 0) pages and takes g_r; F and G are their
// exclusive sums over the requests.  Of count' = count + sum f free pages, the
// j-th from the end is list[count' - 1 - j]: request r's i-th page given back goes
// to j = F_r + i, its i-th taken comes from j = G_r + i, and r is served if G_r +
// g_r <= count'.  So no page waits for another request's; only what is given back
// has to be there before anything is taken, and the tables before the slots.
//
// One cluster of CTAs.  Each works out the sums over all requests for itself (in
// shared memory, a thread having up to 8 requests), then the warps of the cluster
// share the requests, a lane an entry, with a cluster barrier between giving back,
// taking and mapping.
#include <climits>

#include "pages.cuh"

namespace hs {
namespace {

constexpr int TB_NT = 1024, TB_WARPS = TB_NT / 32;
constexpr int MAP_NT = 256, MAP_TOKENS = 2048;      // the mapping launch: tokens a CTA

// n / d for 0 <= n < 2^31, 1 <= d < 2^31, as a product and a shift.
struct Divider {
    uint32_t mul, shift, d;
    explicit Divider(int32_t by)
    {
        d = (uint32_t)by;
        shift = 0;
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int32_t over(int32_t n) const { return (int32_t)((__umulhi(mul, (uint32_t)n) + (uint32_t)n) >> shift); }
};

// A request's page count for its length: what it needs, or -1 if it is left as it is.
__device__ __forceinline__ int32_t pages_needed(const TablesLaunch &a, const Divider &by, int32_t len, int32_t held)
{
    if (len < 0 || held < 0 || held > a.W) return -1;
    const int32_t whole = by.over(len), need = whole + (len - whole * (int32_t)by.d > 0);
    return need <= a.W ? need : -1;
}

// The slot and position of a place: token i of request r, which begins at first.
__device__ __forceinline__ void map_token(const TablesLaunch &a, const Divider &by, int r, int32_t first, int32_t i)
{
    const int32_t len = a.lens[r], held = a.held[r], n = a.new_tokens[r];
    int32_t slot = -1, pos = -1;
    // (a request that is left as it is: its entries do not cover its length)
    if (len >= 0 && n <= len && held >= 0 && held <= a.W && (int64_t)held * a.bs >= len) {
        const int32_t p = len - n + (i - first), b = by.over(p);
        const int32_t page = a.tables[(int64_t)r * a.tables_stride + b];
        const int64_t s = (int64_t)page * a.bs + (p - b * a.bs);
        if (page >= 0 && ((int64_t)page + 1) * a.bs <= kResidentFlag) {
            slot = (int32_t)s;
            pos = p;
        } else if (page >= 0 && a.status) {
            record_status(a.status, r, kStatusBadResident);
        }
    }
    a.slots[i] = slot;
    if (a.positions) a.positions[i] = pos;
}

// The last r in [lo, hi] with first[r] <= i (first[lo] is).
__device__ __forceinline__ int find_request(const int32_t *first, int lo, int hi, int32_t i)
{
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// All that the cluster's CTAs have written is visible to all of them.
__device__ __forceinline__ void cluster_sync(bool alone)
{
    if (alone) {
        __syncthreads();
    } else {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n"
                     "barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

struct Sums {
    int32_t freed, grown;
    int64_t tokens;
};

__device__ __forceinline__ Sums plus(const Sums &x, const Sums &y)
{
    return {x.freed + y.freed, x.grown + y.grown, x.tokens + y.tokens};
}

__device__ __forceinline__ Sums shfl_up(const Sums &x, int d)
{
    return {__shfl_up_sync(0xffffffffu, x.freed, d), __shfl_up_sync(0xffffffffu, x.grown, d),
            __shfl_up_sync(0xffffffffu, x.tokens, d)};
}

// Exclusive sums over the CTA's threads, and all of them in *total.
__device__ Sums scan(const Sums &x, Sums *warp_sums, Sums *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sums y = x;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const Sums z = shfl_up(y, d);
        if (lane >= d) y = plus(y, z);
    }
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    if (warp == 0) {
        Sums w = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const Sums z = shfl_up(w, d);
            if (lane >= d) w = plus(w, z);
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[TB_WARPS - 1];
    const Sums z = shfl_up(y, 1);
    Sums before = {0, 0, 0};
    if (warp > 0) before = warp_sums[warp - 1];
    return lane > 0 ? plus(before, z) : before;
}

// Per request, in shared memory.
struct Request {
    int32_t held, need;      // need -1: left as it is
    int32_t from;            // its first page given back or taken, from the end of the list; -1: none
};

template <bool MAP>
__global__ void __launch_bounds__(TB_NT, 1) tables_kernel(const __grid_constant__ TablesLaunch a, const __grid_constant__ Divider by)
{
    extern __shared__ __align__(16) uint8_t smem[];
    Request *req = reinterpret_cast<Request *>(smem);
    int32_t *first = reinterpret_cast<int32_t *>(req + a.R);      // [R + 1], with MAP
    __shared__ Sums warp_sums[TB_WARPS];
    __shared__ int32_t taken;
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = blockIdx.x, ctas = gridDim.x;
    const bool alone = ctas == 1;
    if (tid == 0) taken = 0;
    after_launch_before();

    // ---- sums over the requests -------------------------------------------------
    const int per = (a.R + TB_NT - 1) / TB_NT, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    Sums mine = {0, 0, 0};
    for (int r = r0; r < r1; ++r) {
        const int32_t len = a.lens[r], held = a.held[r], n = a.new_tokens ? a.new_tokens[r] : 0;
        const int32_t need = pages_needed(a, by, len, held);
        req[r] = {held, need, -1};
        if (need >= 0) {
            const int32_t own = max(need - a.shared_count, 0), had = max(held - a.shared_count, 0);
            mine.freed += max(had - own, 0);
            mine.grown += max(own - had, 0);
        }
        mine.tokens += max(n, 0);
        if (rank == 0 && a.status) {
            if (held < 0 || held > a.W)
                record_status(a.status, r, kStatusBadIndex);
            else if (len >= 0 && need < 0)
                record_status(a.status, r, kStatusBadSeqLen);
            if (n < 0 || n > max(len, 0)) record_status(a.status, r, kStatusBadPosition);
        }
    }
    const int32_t count = min(max(*a.free_count, 0), a.free_capacity);
    Sums total;
    Sums at = scan(mine, warp_sums, &total);
    // (a list without room for all that comes back keeps as much as it holds)
    const int32_t there = (int32_t)min((int64_t)count + total.freed, (int64_t)a.free_capacity);
    for (int r = r0; r < r1; ++r) {
        Request &q = req[r];
        if (q.need >= 0) {
            const int32_t own = max(q.need - a.shared_count, 0), had = max(q.held - a.shared_count, 0);
            if (own <= had) {
                q.from = at.freed;
                at.freed += had - own;
            } else {
                q.from = at.grown;
                at.grown += own - had;
                if (at.grown <= there) {
                    atomicMax(&taken, at.grown);
                } else {
                    q.need = -1;
                    if (rank == 0 && a.status) record_status(a.status, r, kStatusCapacity);
                }
            }
        }
        if (a.new_tokens) {
            const int32_t n = max(a.new_tokens[r], 0), f = (int32_t)min(at.tokens, (int64_t)INT_MAX);
            if (MAP) first[r] = f;
            if (rank == 0) {
                a.offsets[r] = f;
                if (a.status && n > 0 && at.tokens + n > a.tokens) record_status(a.status, r, kStatusCapacity);
            }
            at.tokens += n;
        }
    }
    if (a.new_tokens && tid == 0) {
        const int32_t end = (int32_t)min(total.tokens, (int64_t)INT_MAX);
        if (MAP) first[a.R] = end;
        if (rank == 0) a.offsets[a.R] = end;
    }
    __syncthreads();

    // ---- pages given back ------------------------------------------------------------
    const int warp = rank * TB_WARPS + (tid >> 5), warps = ctas * TB_WARPS;
    if (total.freed > 0 || a.shared_count > 0) {
        for (int r = warp; r < a.R; r += warps) {
            const Request q = req[r];
            if (q.need < 0 || q.need >= q.held) continue;
            int32_t *row = a.tables + (int64_t)r * a.tables_stride;
            for (int32_t e = q.need + lane; e < q.held; e += 32) {
                const int32_t page = row[e], to = there - 1 - (q.from + e - max(q.need, a.shared_count));
                row[e] = -1;
                if (e >= a.shared_count && to >= 0) a.free_list[to] = page;
            }
        }
    }
    // (also: every CTA has read the lengths and counts that are written below)
    cluster_sync(alone);

    // ---- pages taken -----------------------------------------------------------------
    for (int r = warp; r < a.R; r += warps) {
        const Request q = req[r];
        if (q.need < 0) continue;
        int32_t *row = a.tables + (int64_t)r * a.tables_stride;
        for (int32_t e = q.held + lane; e < q.need; e += 32) {
            const int32_t at = there - 1 - (q.from + e - max(q.held, a.shared_count));
            row[e] = e < a.shared_count ? a.shared[e] : a.free_list[at];
        }
        if (lane == 0 && q.need != q.held) a.held[r] = q.need;
    }
    if (rank == 0 && tid == 0) *a.free_count = there - taken;

    // ---- slots -----------------------------------------------------------------------
    if (MAP) {
        cluster_sync(alone);
        const int32_t end = min(first[a.R], a.tokens);
        for (int32_t i = rank * TB_NT + tid; i < a.tokens; i += ctas * TB_NT) {
            if (i < end) {
                const int r = find_request(first, 0, a.R - 1, i);
                map_token(a, by, r, first[r], i);
            } else {
                a.slots[i] = -1;
                if (a.positions) a.positions[i] = -1;
            }
        }
    }
}

// The slots of many tokens, behind tables_kernel: MAP_TOKENS of them a CTA.
__global__ void __launch_bounds__(MAP_NT) map_kernel(const __grid_constant__ TablesLaunch a, const __grid_constant__ Divider by)
{
    after_launch_before();
    const int32_t begin = blockIdx.x * MAP_TOKENS, last = min(a.tokens - begin, MAP_TOKENS) - 1 + begin;
    const int32_t end = min(a.offsets[a.R], a.tokens);
    int lo = 0, hi = 0;
    if (begin < end) {
        lo = find_request(a.offsets, 0, a.R - 1, begin);
        hi = find_request(a.offsets, lo, a.R - 1, min(last, end - 1));
    }
#pragma unroll 4
    for (int32_t i = begin + threadIdx.x; i <= last; i += MAP_NT) {
        if (i < end) {
            const int r = find_request(a.offsets, lo, hi, i);
            map_token(a, by, r, a.offsets[r], i);
        } else {
            a.slots[i] = -1;
            if (a.positions) a.positions[i] = -1;
        }
    }
}

}  // namespace

cudaError_t launch_page_tables(const TablesLaunch &a, cudaStream_t s)
{
    const Divider by(a.bs);
    const bool map = a.new_tokens && a.tokens <= 16384;
    const unsigned ctas = a.R > 32 ? 8 : 1;
    const size_t smem = (size_t)a.R * sizeof(Request) + ((size_t)a.R + 1) * 4;
    auto kernel = map ? tables_kernel<true> : tables_kernel<false>;
    if (smem > 40000) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_behind(kernel, dim3(ctas), TB_NT, smem, ctas, s, a, by);
    if (e != cudaSuccess || !a.new_tokens || map) return e;
    return launch_behind(map_kernel, dim3((a.tokens + MAP_TOKENS - 1) / MAP_TOKENS), MAP_NT, 0, 1, s, a, by);
}

}  // namespace hs
