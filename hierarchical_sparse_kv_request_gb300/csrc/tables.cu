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

// The position of a request's first new token, or LEFT if its tokens have no slots: it is
// left as it is, or they are more than its length.  (held: as the call leaves it)
constexpr int32_t LEFT = INT_MIN;
__device__ __forceinline__ int32_t first_position(const TablesLaunch &a, int32_t len, int32_t held, int32_t n)
{
    return len >= 0 && n <= len && held >= 0 && held <= a.W && (int64_t)held * a.bs >= len ? len - max(n, 0) : LEFT;
}

// The slot and position of token p of request r (p below 0: none), to place i.
__device__ __forceinline__ void map_token(const TablesLaunch &a, const Divider &by, int r, int32_t p, int32_t i)
{
    int32_t slot = -1, pos = -1;
    if (p >= 0) {
        const int32_t b = by.over(p), page = a.tables[(int64_t)r * a.tables_stride + b];
        if (page >= 0 && ((int64_t)page + 1) * a.bs <= kResidentFlag) {
            slot = page * a.bs + (p - b * a.bs);
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

// Pages j of the call from j0 on in steps: eight at a time, so that their loads do not
// wait for one another.
template <class Load, class Store>
__device__ __forceinline__ void move_pages(int32_t j0, int32_t step, int32_t end, Load load, Store store)
{
    constexpr int AT_ONCE = 8;
    for (int32_t j = j0; j < end; j += AT_ONCE * step) {
        int32_t page[AT_ONCE];
        int64_t to[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            if ((int64_t)j + (int64_t)k * step < end) load(j + k * step, page[k], to[k]);
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            if ((int64_t)j + (int64_t)k * step < end) store(page[k], to[k]);
    }
}

// Per request, in shared memory: entries in use and needed (-1: left as it is), the
// first page that it gives back or takes, from the end of the list, its first place and
// the position there.
struct Requests {
    int32_t *held, *need, *freed, *grown, *start, *first;
    __device__ __forceinline__ Requests(uint8_t *smem, int R)
    {
        held = reinterpret_cast<int32_t *>(smem);
        need = held + R;
        freed = need + R;
        grown = freed + R;
        start = grown + R;      // with MAP
        first = start + R;      // [R + 1], with MAP
    }
};
size_t requests_bytes(int R, bool map) { return ((size_t)R * (map ? 6 : 4) + 1) * 4; }

template <bool MAP>
__global__ void __launch_bounds__(TB_NT, 1) tables_kernel(const __grid_constant__ TablesLaunch a, const __grid_constant__ Divider by)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Sums warp_sums[TB_WARPS];
    __shared__ int32_t taken;
    const Requests q(smem, a.R);
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = blockIdx.x, ctas = gridDim.x;
    const bool alone = ctas == 1;
    if (tid == 0) taken = 0;
    after_launch_before();

    // ---- sums over the requests -------------------------------------------------
    const int per = (a.R + TB_NT - 1) / TB_NT, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
    auto own = [&](int32_t n) { return max(n - a.shared_count, 0); };      // of n entries
    Sums mine = {0, 0, 0};
    for (int r = r0; r < r1; ++r) {
        const int32_t len = a.lens[r], held = a.held[r], n = a.new_tokens ? a.new_tokens[r] : 0;
        const int32_t need = pages_needed(a, by, len, held);
        q.held[r] = held;
        q.need[r] = need;
        if (need >= 0) {
            mine.freed += max(own(held) - own(need), 0);
            mine.grown += max(own(need) - own(held), 0);
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
        const int32_t held = q.held[r], need = q.need[r];
        q.freed[r] = at.freed;
        q.grown[r] = at.grown;
        if (need >= 0) {
            const int32_t more = max(own(need) - own(held), 0);
            at.freed += max(own(held) - own(need), 0);
            at.grown += more;
            if (more > 0 && at.grown > there) {
                q.need[r] = -1;
                if (rank == 0 && a.status) record_status(a.status, r, kStatusCapacity);
            } else if (more > 0) {
                atomicMax(&taken, at.grown);
            }
        }
        if (a.new_tokens) {
            const int32_t news = a.new_tokens[r], n = max(news, 0), f = (int32_t)min(at.tokens, (int64_t)INT_MAX);
            if (MAP) {
                q.first[r] = f;
                q.start[r] = first_position(a, a.lens[r], q.need[r] >= 0 ? q.need[r] : held, news);
            }
            if (rank == 0) {
                a.offsets[r] = f;
                if (a.status && n > 0 && at.tokens + n > a.tokens) record_status(a.status, r, kStatusCapacity);
            }
            at.tokens += n;
        }
    }
    if (a.new_tokens && tid == 0) {
        const int32_t end = (int32_t)min(total.tokens, (int64_t)INT_MAX);
        if (MAP) q.first[a.R] = end;
        if (rank == 0) a.offsets[a.R] = end;
    }
    __syncthreads();

    // ---- pages given back: the j-th of all is request r's (j - freed[r])-th -----------------
    const int32_t j0 = rank * TB_NT + tid, step = ctas * TB_NT;
    move_pages(
        j0, step, total.freed,
        [&](int32_t j, int32_t &page, int64_t &to) {
            const int r = find_request(q.freed, 0, a.R - 1, j);
            int32_t *entry = a.tables + (int64_t)r * a.tables_stride + max(q.need[r], a.shared_count) + (j - q.freed[r]);
            page = *entry;
            *entry = -1;
            to = there - 1 - j;
        },
        [&](int32_t page, int64_t to) {
            if (to >= 0) a.free_list[to] = page;
        });
    // entries of the shared prefix, a warp a request
    auto shared_entries = [&](bool back) {
        if (a.shared_count == 0) return;
        for (int r = rank * TB_WARPS + (tid >> 5); r < a.R; r += ctas * TB_WARPS) {
            const int32_t held = q.held[r], need = q.need[r];
            if (need < 0) continue;
            int32_t *row = a.tables + (int64_t)r * a.tables_stride;
            const int32_t from = back ? need : held, to = min(back ? held : need, a.shared_count);
            for (int32_t e = from + lane; e < to; e += 32) row[e] = back ? -1 : a.shared[e];
        }
    };
    shared_entries(true);
    // (also: every CTA has read the lengths and counts that are written below)
    cluster_sync(alone);

    // ---- pages taken -----------------------------------------------------------------
    const int32_t takes = taken;
    move_pages(
        j0, step, takes,
        [&](int32_t j, int32_t &page, int64_t &to) {
            const int r = find_request(q.grown, 0, a.R - 1, j);
            to = (int64_t)r * a.tables_stride + max(q.held[r], a.shared_count) + (j - q.grown[r]);
            page = a.free_list[there - 1 - j];
        },
        [&](int32_t page, int64_t to) { a.tables[to] = page; });
    shared_entries(false);
    if (rank == 0) {
        for (int r = tid; r < a.R; r += TB_NT)
            if (q.need[r] >= 0 && q.need[r] != q.held[r]) a.held[r] = q.need[r];
        if (tid == 0) *a.free_count = there - takes;
    }

    // ---- slots -----------------------------------------------------------------------
    if (MAP) {
        cluster_sync(alone);
        const int32_t end = min(q.first[a.R], a.tokens);
        for (int32_t i = j0; i < a.tokens; i += step) {
            const int r = i < end ? find_request(q.first, 0, a.R - 1, i) : 0;
            const int32_t start = i < end ? q.start[r] : LEFT;
            map_token(a, by, r, start == LEFT ? -1 : start + (i - q.first[r]), i);
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
    auto look = [&](int r) {
        const int32_t start = first_position(a, a.lens[r], a.held[r], a.new_tokens[r]);
        return start == LEFT ? LEFT : start - a.offsets[r];
    };
    if (lo == hi && begin < end) {      // one request (or none behind the last token)
        const int32_t start = look(lo);
#pragma unroll
        for (int k = 0; k < MAP_TOKENS / MAP_NT; ++k) {
            const int32_t i = begin + k * MAP_NT + threadIdx.x;
            if (i <= last) map_token(a, by, lo, i < end && start != LEFT ? start + i : -1, i);
        }
    } else {
#pragma unroll 4
        for (int32_t i = begin + threadIdx.x; i <= last; i += MAP_NT) {
            const int r = i < end ? find_request(a.offsets, lo, hi, i) : 0;
            const int32_t start = i < end ? look(r) : LEFT;
            map_token(a, by, r, start == LEFT ? -1 : start + i, i);
        }
    }
}

}  // namespace

cudaError_t launch_page_tables(const TablesLaunch &a, cudaStream_t s)
{
    const Divider by(a.bs);
    const bool map = a.new_tokens && a.tokens <= 16384;
    const unsigned ctas = a.R > 32 ? 8 : 1;
    const size_t smem = requests_bytes(a.R, map);
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
