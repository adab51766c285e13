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
// One CTA, or one cluster of them.  Each works out the sums over all requests for itself
// (in shared memory, a thread having up to 16 requests), then the warps share the pages
// that come back or go, whichever request's they are, with a barrier between giving back,
// taking and mapping.
//
// Bound by latency: a call's chain is lengths, sums, entries given back, list, entries
// taken and read again for the slots, some 0.4 us each, and the barriers (a cluster's 0.7
// us).  Measured on GB300, GPU time of two calls, one there and one back: 32 requests, up
// to 4 drafted tokens each 6.6 us; 256 requests, 38 of them admitted and 38 finished (some
// 27 thousand pages each way, places for 1.0 M tokens) 22; 128 requests of 2,048 to 81,920
// tokens admitted and finished (43 thousand pages, 2.8 M slots) 21.
#include <atomic>
#include <climits>

#include "pages.cuh"

namespace hs {
namespace {

constexpr int kMostRequests = 8192;                 // HISPARSE_MAX_REQUESTS
constexpr int MAP_NT = 256, MAP_TOKENS = 1024;      // the mapping launch: tokens a CTA (256
                                                    // requests, mixed: 22 us; with a cluster of
                                                    // eight 24, 31 with 4,096)

// n / d for 0 <= n < 2^31, 1 <= d <= 2^30, as a product and a shift; and the last page
// whose rows end below the flag bit.
struct Divider {
    uint32_t mul, shift, d;
    int32_t last_page;
    explicit Divider(int32_t by)
    {
        d = (uint32_t)by;
        shift = 0;
        while ((1ull << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
        last_page = kResidentFlag / by - 1;
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

// The slot and position of token p of request r (p below 0: none), whose table is row,
// to place i.
__device__ __forceinline__ void map_token(const TablesLaunch &a, const Divider &by, int r, const int32_t *row, int32_t p, int32_t i)
{
    int32_t slot = -1, pos = -1;
    if (p >= 0) {
        const int32_t b = by.over(p), page = row[b];
        if ((uint32_t)page <= (uint32_t)by.last_page) {
            slot = p + (page - b) * (int32_t)by.d;
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

// All that the CTAs have written is visible to all of them.
template <int CTAS>
__device__ __forceinline__ void all_sync()
{
    if (CTAS == 1) {
        __syncthreads();
        return;
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// Exclusive sums over the CTA's threads (at most 32 warps), and all of them in *total.
template <int WARPS>
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
        Sums w = {0, 0, 0};
        if (lane < WARPS) w = warp_sums[lane];
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const Sums z = shfl_up(w, d);
            if (lane >= d) w = plus(w, z);
        }
        if (lane < WARPS) warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[WARPS - 1];
    const Sums z = shfl_up(y, 1);
    Sums before = {0, 0, 0};
    if (warp > 0) before = warp_sums[warp - 1];
    return lane > 0 ? plus(before, z) : before;
}

// Pages [0, end) of a call, j of them before request r being first[r]: neighbours, which
// are mostly one request's, a warp, up to eight a lane at a time, so that their loads do
// not wait for one another.
template <class Load, class Store>
__device__ __forceinline__ void move_pages(const int32_t *first, int requests, int warp, int warps, int32_t end, Load load, Store store)
{
    constexpr int AT_ONCE = 8;
    const int lane = threadIdx.x & 31;
    const int32_t a_warp = (int32_t)min(((int64_t)end + warps * 32 - 1) / (warps * 32), (int64_t)AT_ONCE) * 32;
    for (int64_t j0 = (int64_t)warp * a_warp; j0 < end; j0 += (int64_t)warps * a_warp) {
        const int32_t last = (int32_t)min(j0 + a_warp, (int64_t)end) - 1;
        int lo = 0, hi = requests - 1;
        if (a_warp > 32) {
            lo = find_request(first, 0, requests - 1, (int32_t)j0);
            hi = find_request(first, lo, requests - 1, last);
        }
        int32_t page[AT_ONCE];
        int64_t to[AT_ONCE];
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int64_t j = j0 + k * 32 + lane;
            if (j <= last) load(find_request(first, lo, hi, (int32_t)j), (int32_t)j, page[k], to[k]);
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k)
            if (j0 + k * 32 + lane <= last) store(page[k], to[k]);
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

template <int CTAS, int NT, bool MAP>
__global__ void __launch_bounds__(NT, 1) tables_kernel(const __grid_constant__ TablesLaunch a, const __grid_constant__ Divider by)
{
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int WARPS = NT / 32;
    static_assert(WARPS <= 32, "scan");
    __shared__ Sums warp_sums[WARPS];
    __shared__ int32_t taken;
    const Requests q(smem, a.R);
    const int tid = threadIdx.x, lane = tid & 31;
    const int rank = blockIdx.x;
    if (tid == 0) taken = 0;
    after_launch_before();
    // map_kernel may be placed now, as it waits before it does anything.  (Not so the
    // caller's next launch, where none follows: a swap-in may read its resident tables
    // ahead of its wait, see hisparse_set_programmatic_launch.)
    if (!MAP && a.new_tokens) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- sums over the requests -------------------------------------------------
    const int per = (a.R + NT - 1) / NT, r0 = min(tid * per, a.R), r1 = min(r0 + per, a.R);
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
    Sums at = scan<WARPS>(mine, warp_sums, &total);
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
    const int warp = rank * WARPS + (tid >> 5), warps = CTAS * WARPS;
    move_pages(
        q.freed, a.R, warp, warps, total.freed,
        [&](int r, int32_t j, int32_t &page, int64_t &to) {
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
        for (int r = warp; r < a.R; r += warps) {
            const int32_t held = q.held[r], need = q.need[r];
            if (need < 0) continue;
            int32_t *row = a.tables + (int64_t)r * a.tables_stride;
            const int32_t from = back ? need : held, to = min(back ? held : need, a.shared_count);
            for (int32_t e = from + lane; e < to; e += 32) row[e] = back ? -1 : a.shared[e];
        }
    };
    shared_entries(true);
    // (also: every CTA has read the lengths and counts that are written below)
    all_sync<CTAS>();

    // ---- pages taken -----------------------------------------------------------------
    const int32_t takes = taken;
    move_pages(
        q.grown, a.R, warp, warps, takes,
        [&](int r, int32_t j, int32_t &page, int64_t &to) {
            to = (int64_t)r * a.tables_stride + max(q.held[r], a.shared_count) + (j - q.grown[r]);
            page = a.free_list[there - 1 - j];
        },
        [&](int32_t page, int64_t to) { a.tables[to] = page; });
    shared_entries(false);
    if (rank == 0) {
        for (int r = tid; r < a.R; r += NT)
            if (q.need[r] >= 0 && q.need[r] != q.held[r]) a.held[r] = q.need[r];
        if (tid == 0) *a.free_count = there - takes;
    }

    // ---- slots -----------------------------------------------------------------------
    if (MAP) {
        all_sync<CTAS>();
        const int32_t end = min(q.first[a.R], a.tokens);
        for (int32_t i = rank * NT + tid; i < a.tokens; i += CTAS * NT) {
            const int r = i < end ? find_request(q.first, 0, a.R - 1, i) : 0;
            const int32_t start = i < end ? q.start[r] : LEFT;
            map_token(a, by, r, a.tables + (int64_t)r * a.tables_stride, start == LEFT ? -1 : start + (i - q.first[r]), i);
        }
    }
}

// The slots of many tokens, behind tables_kernel: MAP_TOKENS of them a CTA.
__global__ void __launch_bounds__(MAP_NT) map_kernel(const __grid_constant__ TablesLaunch a, const __grid_constant__ Divider by)
{
    __shared__ int32_t sums[2][MAP_NT / 32];
    const int32_t begin = blockIdx.x * MAP_TOKENS, last = min(a.tokens - begin, MAP_TOKENS) - 1 + begin;
    after_launch_before();
    const int32_t end = min(a.offsets[a.R], a.tokens);
    // The requests of the first and the last token: as many as begin at or before them,
    // counted by all threads at once (a search: 9 to 13 loads one behind the other).
    int lo = 0, hi = 0;
#pragma unroll 4
    for (int r = threadIdx.x; r < a.R; r += MAP_NT) {
        const int32_t first = a.offsets[r];
        lo += first <= begin;
        hi += first <= min(last, end - 1);
    }
    lo = __reduce_add_sync(0xffffffffu, lo);
    hi = __reduce_add_sync(0xffffffffu, hi);
    if ((threadIdx.x & 31) == 0) {
        sums[0][threadIdx.x >> 5] = lo;
        sums[1][threadIdx.x >> 5] = hi;
    }
    __syncthreads();
    lo = hi = -1;
#pragma unroll
    for (int k = 0; k < MAP_NT / 32; ++k) {
        lo += sums[0][k];
        hi += sums[1][k];
    }
    auto look = [&](int r) {
        const int32_t start = first_position(a, a.lens[r], a.held[r], a.new_tokens[r]);
        return start == LEFT ? LEFT : start - a.offsets[r];
    };
    if (lo == hi && begin < end) {      // one request (or none behind the last token)
        const int32_t start = look(lo);
        const int32_t *row = a.tables + (int64_t)lo * a.tables_stride;
#pragma unroll
        for (int k = 0; k < MAP_TOKENS / MAP_NT; ++k) {
            const int32_t i = begin + k * MAP_NT + threadIdx.x;
            if (i <= last) map_token(a, by, lo, row, i < end && start != LEFT ? start + i : -1, i);
        }
    } else {
#pragma unroll 4
        for (int32_t i = begin + threadIdx.x; i <= last; i += MAP_NT) {
            const int r = i < end ? find_request(a.offsets, lo, hi, i) : 0;
            const int32_t start = i < end ? look(r) : LEFT;
            map_token(a, by, r, a.tables + (int64_t)r * a.tables_stride, start == LEFT ? -1 : start + i, i);
        }
    }
}

}  // namespace

// Sets a kernel's attributes on the current device, once.
template <int CTAS, int NT, bool MAP>
static cudaError_t prepare_tables()
{
    constexpr int kDevices = 64;
    static std::atomic<bool> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (known[dev].load(std::memory_order_acquire)) return cudaSuccess;
    auto kernel = tables_kernel<CTAS, NT, MAP>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)requests_bytes(kMostRequests, MAP));
    if (e == cudaSuccess && CTAS > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) known[dev].store(true, std::memory_order_release);
    return e;
}

template <int CTAS, int NT, bool MAP>
static cudaError_t launch_tables(const TablesLaunch &a, const Divider &by, cudaStream_t s)
{
    const cudaError_t e = prepare_tables<CTAS, NT, MAP>();
    if (e != cudaSuccess) return e;
    return launch_behind(tables_kernel<CTAS, NT, MAP>, dim3(CTAS), NT, requests_bytes(a.R, MAP), CTAS, s, a, by);
}

// One CTA for a decode step, a cluster of sixteen where many pages may come and go.  What a
// call moves is known on the device alone; on the host, that a step has few tokens (or, where
// none are placed, few requests), and that it moves no more pages than the tables hold
// behind the shared prefix.  GPU time of a call there and one back, one CTA and the cluster:
// up to 4 tokens more for 32 requests of 626 pages each 7.9 and 9.0 us, for 256 of 626 9.0 and
// 9.7; 4 of those 256 finished and back 15.7 and 12.5; all 32 finished and back 37 and
// 10.7, 32 of 1,281 pages 64 and 11.6, of 81,921 3,495 and 162.  (Prompts: 128 requests of 2,048
// to 81,920 tokens 90 us and 20.8, 23.2 with eight CTAs of 1,024 threads.)
constexpr int64_t kStepPages = 32768;
static bool one_cta(const TablesLaunch &a)
{
    if ((int64_t)a.R * (a.W - a.shared_count) > kStepPages) return false;
    return a.new_tokens ? a.R <= 256 && a.tokens <= 4096 : a.R <= 32;
}

cudaError_t launch_page_tables(const TablesLaunch &a, cudaStream_t s)
{
    const Divider by(a.bs);
    // Few slots in the same launch (1.0 M in one: 69 us for 256 requests with a
    // cluster of eight, 25 in two).
    const bool map = a.new_tokens && a.tokens <= 16384;
    const bool step = one_cta(a);
    const cudaError_t e = step ? map ? launch_tables<1, 256, true>(a, by, s) : launch_tables<1, 256, false>(a, by, s)
                               : map ? launch_tables<16, 512, true>(a, by, s) : launch_tables<16, 512, false>(a, by, s);
    if (e != cudaSuccess || !a.new_tokens || map || a.tokens == 0) return e;
    return launch_behind(map_kernel, dim3((a.tokens + MAP_TOKENS - 1) / MAP_TOKENS), MAP_NT, 0, 1, s, a, by);
}

}  // namespace hs
