// prefix.cu -- attention of a whole batch over a prefix that its requests share
// (include/hisparse_pages.h, hisparse_attend_prefix).
//
// The mathematics.  The heads of all requests are the rows of one matrix Q (M = R
// H rows of 576).  With s = scale * log2(e) * (q . row), a running reference m of
// the row maximum, l = sum 2^(s - m) and O = sum 2^(s - m) * latent over the rows
// seen so far; when s outgrows m by more than 8, m moves and l and O are
// multiplied by 2^(m_old - m_new).  A part comes in as one more row of score
// part_lse * log2(e) and value part.  out = O / l, lse = (m + log2 l) ln 2.
//
// Three launches.  expand_kernel reads the prefix's pages once and writes its rows
// to the workspace in 16 bits, in the layout that the tensor cores read, so that
// tiles come in as plain bulk copies whatever the format, the pages' size and the
// strides; rows that are not there are 0, and a bit a row says so.  prefix_kernel
// multiplies.  join_kernel adds up heads whose rows were split.
//
// prefix_kernel.  O of 128 heads by 512 values would fill tensor memory and leave
// nothing for S, and 64 heads a CTA run the tensor cores at half their rate (128
// rows of keys by 64 heads: 4,364 cycles).  So a pair of CTAs works on one product
// (cta_group::2, M = 128), each with 64 heads: a CTA's rows of D are spread over
// all 128 lanes, the first half of the columns in lanes 0-63 and the second in
// 64-127, and O takes 256 columns, S of 128 keys 64.  Both products run at the full
// rate (2,184 cycles a tile of 128 keys, measured).  Of the keys of a tile and of
// the values each CTA has half in the role of B: in S = Q K^T its own 64 keys, all
// 576 values; in O += P V all keys, its own 256 values.  So a quarter of the tile is
// used twice in one CTA, and 32 KB more come in for the second product, where the
// first has freed shared memory:
//   slots of 16 KB (64 keys by 128 values), four a tile, X0 Y0 X1 Y1, in a ring of
//   ten; X_h are values 128 h, Y_h values 256 + 128 h and on, of the CTA's own keys.
//   After S the first CTA keeps X and gets, in Y, the other CTA's keys of its
//   values X; the second keeps Y and gets, in X, the first one's keys of Y.  A
//   descriptor is one for both CTAs: at X_h both have keys 0-63, at Y_h 64-127.
//   The rope part (8 KB) has a ring of three.
// The queries do not fit either shared memory or what O and S leave of tensor
// memory (192 columns): 384 of their values are there, in both halves of the lanes,
// the other 192 in shared memory.
//   warps 0-3  softmax: a thread a lane, that is a head and half of the tile's keys;
//   warp 4     brings keys in, warp 5 the values of the other CTA's keys;
//   warp 6     of the first CTA issues the MMAs, S of the next tile ahead of O of
//              this one; that of the second says what has come in there.
// The heads' tiles in a row are cut evenly among the pairs, wherever a head ends.
#include <atomic>
#include <mutex>

#include "pages.cuh"

namespace hs {
namespace {

constexpr int PAIR_HEADS = 128, CTA_HEADS = 64, KEYS = 128;
constexpr int MAX_PAIRS = 76;                    // pairs of SMs of a GB300
constexpr uint32_t BLOCK = 64 * 128;             // 64 values of 64 keys, swizzled
constexpr uint32_t SLOT = 2 * BLOCK;
constexpr uint32_t HALF_TILE = 9 * BLOCK;        // 64 keys: X0 Y0 X1 Y1 rope
constexpr uint32_t TILE_BYTES = 2 * HALF_TILE;
constexpr int SLOTS = 10, ROPES = 3;
constexpr int Q_TMEM = 6, Q_SMEM = 9 - Q_TMEM;   // blocks of the queries

constexpr uint32_t ROPE_AT = SLOTS * SLOT, Q_AT = ROPE_AT + ROPES * BLOCK, P_AT = Q_AT + Q_SMEM * BLOCK;
constexpr uint32_t MISC_AT = P_AT + 2 * BLOCK;
constexpr int PX_NT = 256, SOFTMAX = 4, KEY_WARP = 4, VALUE_WARP = 5, MMA_WARP = 6;

// columns of tensor memory
constexpr uint32_t T_O = 0, T_S = 256, T_Q = 320;

struct PrefixSmem {
    uint64_t keys[SLOTS], ropes[ROPES], values[4];      // arrived (in the first CTA: in both)
    uint64_t slot_free[SLOTS], rope_free[ROPES];        // the products that read it are done
    uint64_t scored[2], added;                          // S is there; O is
    uint64_t queries, read, weighed;                    // (in the first CTA, from both) Q is there, S read, P there
    uint64_t drained;
    uint32_t tmem;
    int gave_up;
    float top[2][2][CTA_HEADS];      // [tile % 2][half of the keys]
    float sum[2][CTA_HEADS];
};
constexpr size_t PX_SMEM = MISC_AT + sizeof(PrefixSmem);
static_assert(PX_SMEM <= 232448, "shared memory of a CTA");

// The latent block (of 64 values; 8: the rope part) at place n of a half tile.
__host__ __device__ constexpr int block_at(int n) { return n == 8 ? 8 : (n >> 2) * 2 + (n >> 1 & 1) * 4 + (n & 1); }

// How a call is cut up, and its workspace.
struct PrefixParts {
    int tiles;               // of 128 keys
    int groups;              // of 128 heads
    int pairs;
    int64_t units;           // tiles * groups; pair p takes units p * units / pairs to (p + 1) * units / pairs
    uint8_t *image;          // [tiles][2] half tiles
    uint32_t *there;         // [tiles][4] a bit a key
    float *o;                // [pairs][2][128][512]: parts of heads that a pair does not have whole
    float2 *ml;              // [pairs][2][128] reference and sum
};

__host__ __device__ __forceinline__ int64_t first_unit(const PrefixParts &w, int pair) { return w.units * pair / w.pairs; }

// The pair that has a unit.
__host__ __device__ __forceinline__ int pair_of(const PrefixParts &w, int64_t unit)
{
    int p = (int)(((unit + 1) * w.pairs - 1) / w.units);
    return p;
}

// ---- expand ------------------------------------------------------------------------

constexpr int EX_NT = 256, EX_KEYS = 32, EX_ROWS = EX_KEYS / (EX_NT / 32);

template <int DT, int ROW>
__global__ void __launch_bounds__(EX_NT) expand_kernel(const __grid_constant__ PrefixLaunch a, const __grid_constant__ PrefixParts w)
{
    __shared__ uint32_t there;
    __shared__ int bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) there = 0, bad = 0;
    __syncthreads();
    after_launch_before();
    const int t0 = blockIdx.x * EX_KEYS + warp * EX_ROWS;
    int64_t row = -1;
    if (lane < EX_ROWS && t0 + lane < a.len) {
        const int t = t0 + lane, b = t / a.bs;
        const int32_t page = a.table[b];
        row = (int64_t)page * a.bs + (t - b * a.bs);
        if (page < 0 || row >= a.num_rows) {
            row = -1;
            if (page != -1) bad = 1;
        }
    }
    const uint32_t named = __ballot_sync(0xffffffffu, row >= 0);
    uint4 v[EX_ROWS][2], rope[EX_ROWS];
#pragma unroll
    for (int j = 0; j < EX_ROWS; ++j) {
        const int64_t n = __shfl_sync(0xffffffffu, row, j);
        v[j][0] = v[j][1] = rope[j] = make_uint4(0, 0, 0, 0);
        if (n >= 0) {
            const uint8_t *p = a.rows + n * a.row_stride;
            v[j][0] = load_latent8<DT, ROW>(p, lane);
            v[j][1] = load_latent8<DT, ROW>(p, lane + 32);
            if (lane < 8) rope[j] = ld_dev_v4(p + rope_at(ROW) + lane * 16);
        }
    }
#pragma unroll
    for (int j = 0; j < EX_ROWS; ++j) {
        const int t = t0 + j, i = t & 63;
        uint8_t *half = w.image + (int64_t)(t >> 6) * HALF_TILE;
        const uint32_t u = ((lane & 7) ^ (i & 7)) << 4;
        // unit lane + 32 k is in block lane / 8 + 4 k, which is at place 0 1 4 5, 2 3 6 7
        const int place = (lane >> 4) * 4 + (lane >> 3 & 1);
        st_v4(half + place * BLOCK + i * 128 + u, v[j][0]);
        st_v4(half + (place + 2) * BLOCK + i * 128 + u, v[j][1]);
        if (lane < 8) st_v4(half + 8 * BLOCK + i * 128 + u, rope[j]);
    }
    if (lane == 0) atomicOr(&there, named << (warp * EX_ROWS));
    __syncthreads();
    if (threadIdx.x == 0) w.there[blockIdx.x] = there;
    if (bad && a.status)
        for (int r = threadIdx.x; r < a.R; r += EX_NT) record_status(a.status, r, kStatusBadResident);
}

// ---- pairs of CTAs ---------------------------------------------------------------

__device__ __forceinline__ void arrive_in(uint32_t bar)      // in any CTA of the cluster
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool try_acquire(uint32_t bar, uint32_t parity)      // what another CTA has released
{
    uint32_t ok;
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                 "selp.u32 %0, 1, 0, p;\n"
                 "}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ bool wait_acquire(uint32_t bar, uint32_t parity, volatile int *gave_up)
{
    if (try_acquire(bar, parity)) return true;
    return mbar_wait_long(bar, parity, gave_up) && try_acquire(bar, parity);
}

__device__ __forceinline__ void pair_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
                 "}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

// With A in tensor memory: row i in lanes i and i + 64.
__device__ __forceinline__ void pair_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n"
                 ".reg .pred p;\n"
                 "setp.ne.u32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n"
                 "}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                 : "memory");
}

// Arrive on this mbarrier of both CTAs once every MMA this thread has issued is done.
__device__ __forceinline__ void pair_commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void bring(uint32_t dst, const uint8_t *src, uint32_t bytes, uint32_t bar)
{
    mbar_expect(bar, bytes);
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// 32 columns of the thread's lane.
__device__ __forceinline__ void tmem_ld_32(uint32_t at, uint32_t (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 " HS_REGS32 ", [%32];"
                 : HS_R4(v, 0), HS_R4(v, 4), HS_R4(v, 8), HS_R4(v, 12), HS_R4(v, 16), HS_R4(v, 20), HS_R4(v, 24), HS_R4(v, 28)
                 : "r"(at));
}

__device__ __forceinline__ void tmem_st_32(uint32_t at, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], " HS_REGS32 ";" ::HS_I4(v, 0), HS_I4(v, 4), HS_I4(v, 8), HS_I4(v, 12),
                 HS_I4(v, 16), HS_I4(v, 20), HS_I4(v, 24), HS_I4(v, 28), "r"(at)
                 : "memory");
}

// A part as one more row: its weight against reference m and sum l, which move.
// Returns what O has to be multiplied by.
__device__ __forceinline__ float add_part(float &m, float &l, float part_lse, float *weight)
{
    const float s = part_lse * kLog2e, n = s > m ? s : m;      // (a NaN does not move m)
    const float f = n == -INFINITY ? 1.0f : ex2(m - n);
    *weight = n == -INFINITY ? 0.0f : ex2(s - n);
    if (s != s) *weight = s;
    m = n;
    l = l * f + *weight;
    return f;
}

// Where a head's values go, or come from.
struct HeadPlace {
    int r, h;
    int64_t n;
    __device__ __forceinline__ HeadPlace(const PrefixLaunch &a, int64_t row) : r((int)(row / a.H)), h((int)(row - (int64_t)r * a.H)), n(row) {}
};

template <int DT>
__device__ __forceinline__ uint4 weighted8(const float (&o)[8], float f, uint4 part, float weight, bool joined)
{
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = o[j] * f;
    if (joined) {
        const uint32_t p[4] = {part.x, part.y, part.z, part.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = pair_to_float<DT>(p[j]);
            x[2 * j] = fmaf(v.x, weight, x[2 * j]);
            x[2 * j + 1] = fmaf(v.y, weight, x[2 * j + 1]);
        }
    }
    return make_uint4(floats_to_pair<DT>(x[0], x[1]), floats_to_pair<DT>(x[2], x[3]), floats_to_pair<DT>(x[4], x[5]),
                      floats_to_pair<DT>(x[6], x[7]));
}

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PX_NT, 1)
    prefix_kernel(const __grid_constant__ PrefixLaunch a, const __grid_constant__ PrefixParts w)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    PrefixSmem &sm = *reinterpret_cast<PrefixSmem *>(smem + MISC_AT);
    const uint32_t base = smem_u32(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1;
    const int64_t u0 = first_unit(w, pair), u1 = first_unit(w, pair + 1);
    const int count = (int)(u1 - u0);      // tiles of this pair, over all its groups of heads
    auto bar = [](const uint64_t &b) { return smem_u32(&b); };

    if (warp == MMA_WARP) {
        if (lane == 0) {
            const int both = rank == 0 ? 2 : 1;      // the first CTA also hears of the second
            for (int s = 0; s < SLOTS; ++s) mbar_init(bar(sm.keys[s]), both), mbar_init(bar(sm.slot_free[s]), 1);
            for (int s = 0; s < ROPES; ++s) mbar_init(bar(sm.ropes[s]), both), mbar_init(bar(sm.rope_free[s]), 1);
            for (int s = 0; s < 4; ++s) mbar_init(bar(sm.values[s]), both);
            mbar_init(bar(sm.scored[0]), 1);
            mbar_init(bar(sm.scored[1]), 1);
            mbar_init(bar(sm.added), 1);
            mbar_init(bar(sm.queries), 2 * SOFTMAX);
            mbar_init(bar(sm.read), 2 * SOFTMAX);
            mbar_init(bar(sm.weighed), 2 * SOFTMAX);
            mbar_init(bar(sm.drained), 1);
            sm.gave_up = 0;
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        }
        __syncwarp();
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&sm.tmem)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    pair_sync();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    volatile int *gave_up = &sm.gave_up;
    auto all = [](bool ok) { return __all_sync(0xffffffffu, ok) != 0; };
    bool ok = true;
    after_launch_before();

    if (warp == KEY_WARP) {
        // ---- this CTA's keys of every tile ------------------------------------------
        int slot = 0, rope = 0, n = 0, tile = (int)(u0 % w.tiles);
        uint32_t slot_phase = 1, rope_phase = 1;      // (nothing to wait for the first time round)
        for (; ok && n < count; ++n) {
            const uint8_t *src = w.image + ((int64_t)tile * 2 + rank) * HALF_TILE;
            for (int p = 0; ok && p < 4; ++p) {
                if (!(ok = all(mbar_wait(bar(sm.slot_free[slot]), slot_phase, gave_up)))) break;
                if (elect_one()) bring(base + slot * SLOT, src + p * SLOT, SLOT, bar(sm.keys[slot]));
                __syncwarp();
                if (++slot == SLOTS) slot = 0, slot_phase ^= 1;
            }
            if (!ok || !(ok = all(mbar_wait(bar(sm.rope_free[rope]), rope_phase, gave_up)))) break;
            if (elect_one()) bring(base + ROPE_AT + rope * BLOCK, src + 4 * SLOT, BLOCK, bar(sm.ropes[rope]));
            __syncwarp();
            if (++rope == ROPES) rope = 0, rope_phase ^= 1;
            if (++tile == w.tiles) tile = 0;
        }
    } else if (warp == VALUE_WARP) {
        // ---- the other CTA's keys, for this one's values --------------------------------
        int slot = rank == 0 ? 1 : 0, tile = (int)(u0 % w.tiles);      // Y0 or X0
        for (int n = 0; ok && n < count; ++n) {
            if (!(ok = all(mbar_wait(bar(sm.scored[n & 1]), (n >> 1) & 1, gave_up)))) break;
            const uint8_t *src = w.image + ((int64_t)tile * 2 + (rank ^ 1)) * HALF_TILE + rank * SLOT;
            if (elect_one())
                for (int h = 0; h < 2; ++h) {
                    int s = slot + 2 * h;
                    if (s >= SLOTS) s -= SLOTS;
                    bring(base + s * SLOT, src + h * 2 * SLOT, SLOT, bar(sm.values[(n & 1) * 2 + h]));
                }
            __syncwarp();
            slot += 4;
            if (slot >= SLOTS) slot -= SLOTS;
            if (++tile == w.tiles) tile = 0;
        }
    } else if (warp == MMA_WARP && rank == 1) {
        // ---- what has come in here, to the first CTA --------------------------------------
        int slot = 0, rope = 0, tile = (int)(u0 % w.tiles);
        uint32_t slot_phase = 0, rope_phase = 0;
        auto tell = [&](const uint64_t &b, uint32_t phase) {
            if (!(ok = ok && all(mbar_wait(bar(b), phase, gave_up)))) return;
            if (lane == 0) arrive_in(in_cta(bar(b), 0));
        };
        auto keys = [&]() {
            for (int p = 0; p < 4; ++p) {
                tell(sm.keys[slot], slot_phase);
                if (++slot == SLOTS) slot = 0, slot_phase ^= 1;
            }
            tell(sm.ropes[rope], rope_phase);
            if (++rope == ROPES) rope = 0, rope_phase ^= 1;
        };
        bool ahead = false;      // the keys of tile n have been told of
        for (int n = 0; ok && n < count; ++n) {
            if (!ahead) keys();
            ahead = n + 1 < count && tile + 1 < w.tiles;
            if (ahead) keys();
            for (int h = 0; h < 2; ++h) tell(sm.values[(n & 1) * 2 + h], (n >> 1) & 1);
            if (++tile == w.tiles) tile = 0;
        }
    } else if (warp == MMA_WARP) {
        // ---- MMA issue ------------------------------------------------------------------
        constexpr uint32_t qk = mma_desc(128, KEYS, DT == kBf16, false), pv = mma_desc(128, 256, DT == kBf16, true);
        int slot = 0, rope = 0, tile = (int)(u0 % w.tiles), group = 0;
        uint32_t slot_phase = 0, rope_phase = 0;
        auto wait = [&](const uint64_t &b, uint32_t phase) {
            ok = ok && all(wait_acquire(bar(b), phase, gave_up));
            return ok;
        };
        auto scores = [&](int n) {            // S = Q K^T of tile n
            if (n > 0 && !wait(sm.read, (n - 1) & 1)) return;
            uint32_t q_col = tmem + T_Q;
            uint64_t q_desc = smem_desc(base + Q_AT, 16, 1024);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                if (!wait(sm.keys[slot], slot_phase)) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t k_desc = smem_desc(base + slot * SLOT, 16, 1024);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {      // 16 values a step: 32 bytes, 8 columns
                        const uint64_t k = k_desc + (x >> 2) * (BLOCK >> 4) + (x & 3) * 2;
                        if (p < Q_TMEM / 2)
                            pair_mma_ts(tmem + T_S, q_col + x * 8, k, qk, p + x > 0);
                        else
                            pair_mma(tmem + T_S, q_desc + (x >> 2) * (BLOCK >> 4) + (x & 3) * 2, k, qk, true);
                    }
                }
                __syncwarp();
                q_col += 64;
                if (++slot == SLOTS) slot = 0, slot_phase ^= 1;
            }
            if (!wait(sm.ropes[rope], rope_phase)) return;
            tc_fence_after();
            if (elect_one()) {
                const uint64_t k_desc = smem_desc(base + ROPE_AT + rope * BLOCK, 16, 1024);
                q_desc += 2 * (BLOCK >> 4);
#pragma unroll
                for (int x = 0; x < 4; ++x) pair_mma(tmem + T_S, q_desc + x * 2, k_desc + x * 2, qk, true);
                pair_commit(bar(sm.scored[n & 1]));
                pair_commit(bar(sm.rope_free[rope]));
            }
            __syncwarp();
            if (++rope == ROPES) rope = 0, rope_phase ^= 1;
        };
        int v_slot = 0;
        bool ahead = false, begins = true;
        for (int n = 0; ok && n < count; ++n) {
            if (begins) {
                if (!wait(sm.queries, group & 1)) break;
                ++group;
            }
            if (!ahead) scores(n);
            ahead = n + 1 < count && tile + 1 < w.tiles;
            if (ok && ahead) scores(n + 1);
            if (!ok || !wait(sm.weighed, n & 1)) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {            // O += P V, 256 values
                if (!wait(sm.values[(n & 1) * 2 + h], (n >> 1) & 1)) break;
                tc_fence_after();
                const int x_slot = v_slot, y_slot = v_slot + 1;      // (the ring has an even number of them)
                if (elect_one()) {
                    const uint64_t p_desc = smem_desc(base + P_AT, 16, 1024);
                    const uint64_t x_desc = smem_desc(base + x_slot * SLOT, BLOCK, 1024);
                    const uint64_t y_desc = smem_desc(base + y_slot * SLOT, BLOCK, 1024);
#pragma unroll
                    for (int x = 0; x < 8; ++x)      // 16 keys a step
                        pair_mma(tmem + T_O + h * 128, p_desc + (x >> 2) * (BLOCK >> 4) + (x & 3) * 2,
                                 (x < 4 ? x_desc : y_desc) + (x & 3) * (2048 >> 4), pv, !begins || x > 0);
                    pair_commit(bar(sm.slot_free[x_slot]));
                    pair_commit(bar(sm.slot_free[y_slot]));
                    if (h == 1) pair_commit(bar(sm.added));
                }
                __syncwarp();
                v_slot += 2;
                if (v_slot == SLOTS) v_slot = 0;
            }
            begins = ++tile == w.tiles;
            if (begins) tile = 0;
        }
        if (!ok) {     // let what was issued end before the pair goes
            if (elect_one()) pair_commit(bar(sm.drained));
            for (int i = 0; i < (1 << 20) && !mbar_try(bar(sm.drained), 0); ++i) {}
        }
        __syncwarp();
    } else if (warp < SOFTMAX) {
        // ---- softmax: a thread has head (warp % 2) 32 + lane of the CTA's, and half of
        // the keys, and in the end half of the values -----------------------------------
        const int i = (warp & 1) * 32 + lane, half = warp >> 1;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const uint32_t queries_at = in_cta(bar(sm.queries), 0), read_at = in_cta(bar(sm.read), 0), weighed_at = in_cta(bar(sm.weighed), 0);
        auto tell = [&](uint32_t at) {
            __syncwarp();
            if (lane == 0) arrive_in(at);
        };
        // With the warp that has the heads' other half: whether both go on.  (Nothing
        // limits this wait: both warps come here, whatever has gone wrong.)
        auto meet = [&](bool go) {
            uint32_t both;
            asm volatile("{\n"
                         ".reg .pred p, q;\n"
                         "setp.ne.u32 p, %1, 0;\n"
                         "barrier.cta.red.and.pred q, %2, 64, p;\n"
                         "selp.u32 %0, 1, 0, q;\n"
                         "}"
                         : "=r"(both)
                         : "r"((uint32_t)go), "r"(1 + (warp & 1))
                         : "memory");
            return both != 0;
        };
        // (scale 0: not 0 times the -inf of a row that is not there)
        const bool nan = a.scale != a.scale;
        const float f = nan ? 1.0f : fmaxf(fabsf(a.scale) * kLog2e, FLT_MIN);
        int n = 0;
        int64_t u = u0;
        for (int part = 0; ok && u < u1; ++part) {
            const int group = (int)(u / w.tiles), t0 = (int)(u - (int64_t)group * w.tiles);
            const int t1 = (int)min((int64_t)w.tiles, t0 + (u1 - u));
            u += t1 - t0;
            const int64_t head = (int64_t)group * PAIR_HEADS + rank * CTA_HEADS + i;
            const bool on = head < (int64_t)a.R * a.H;
            const HeadPlace at(a, on ? head : 0);
            {      // the queries, with the sign of the scale (or NaN)
                const uint8_t *q = a.q + at.r * a.q_rs + at.h * a.q_hs;
                const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u, set = nan ? 0x7FFF7FFFu : 0u;
                auto load = [&](int unit) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (on) v = ld_dev_v4(q + unit * 16);
                    return make_uint4((v.x ^ flip) | set, (v.y ^ flip) | set, (v.z ^ flip) | set, (v.w ^ flip) | set);
                };
#pragma unroll
                for (int b = 0; b < Q_TMEM; ++b) {
                    uint32_t v[32];
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        const uint4 y = load(block_at(b) * 8 + x);
                        v[4 * x] = y.x, v[4 * x + 1] = y.y, v[4 * x + 2] = y.z, v[4 * x + 3] = y.w;
                    }
                    tmem_st_32(lanes + T_Q + b * 32, v);
                }
#pragma unroll
                for (int b = 0; b < Q_SMEM; ++b)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {      // (each of a head's two threads half of it)
                        const int unit = half * 4 + x;
                        st_smem_v4(base + Q_AT + b * BLOCK + i * 128 + ((unit ^ (i & 7)) << 4), load(block_at(Q_TMEM + b) * 8 + unit));
                    }
                tmem_wait_st();
                fence_async_smem();
                tc_fence_before();
                tell(queries_at);
            }
            float m = -INFINITY, l = 0.0f;
            const uint32_t *there = w.there + half * 2;
            uint2 next = *reinterpret_cast<const uint2 *>(there + (int64_t)t0 * 4);
            for (int t = t0; t < t1; ++t, ++n) {
                const uint2 named = next;
                if (t + 1 < t1) next = *reinterpret_cast<const uint2 *>(there + (int64_t)(t + 1) * 4);
                ok = ok && all(mbar_wait(bar(sm.scored[n & 1]), (n >> 1) & 1, gave_up));
                tc_fence_after();
                uint32_t v[2][32];
                tmem_ld_32(lanes + T_S, v[0]);
                tmem_ld_32(lanes + T_S + 32, v[1]);
                tmem_wait_ld();
                tc_fence_before();
                tell(read_at);
                float (&x)[2][32] = reinterpret_cast<float (&)[2][32]>(v);
                if ((named.x & named.y) != 0xFFFFFFFFu) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        if (!(named.x >> j & 1u)) x[0][j] = -INFINITY;
                        if (!(named.y >> j & 1u)) x[1][j] = -INFINITY;
                    }
                }
                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    top[0] = fmaxf(top[0], x[0][j]);
                    top[1] = fmaxf(top[1], x[0][j + 1]);
                    top[2] = fmaxf(top[2], x[1][j]);
                    top[3] = fmaxf(top[3], x[1][j + 1]);
                }
                float s = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
                sm.top[n & 1][half][i] = s;
                if (!(ok = meet(ok))) break;
                s = fmaxf(s, sm.top[n & 1][half ^ 1][i]);
                float d = 1.0f;
                const bool moves = __any_sync(0xffffffffu, s > m + kMoveAbove);
                if (moves) {
                    const float to = fmaxf(m, s);
                    d = to == -INFINITY ? 1.0f : ex2(m - to);
                    m = to;
                    l *= d;
                }
                const float r = m == -INFINITY ? 0.0f : -m;
                float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float p0 = ex2(fmaf(x[k][j], f, r)), p1 = ex2(fmaf(x[k][j + 1], f, r));
                        sum[(j >> 1) & 3] += p0 + p1;
                        v[k][j >> 1] = floats_to_pair<DT>(p0, p1);
                    }
                l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                // P and O are free once the product before is done
                if (n > 0 && !(ok = all(mbar_wait(bar(sm.added), (n - 1) & 1, gave_up)))) continue;
                if (moves && t > t0) {
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        uint32_t o[32];
                        tmem_ld_32(lanes + T_O + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * d);
                        tmem_st_32(lanes + T_O + c, o);
                    }
                    tmem_wait_st();
                }
                const uint32_t p_at = base + P_AT + half * BLOCK + i * 128;
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int x4 = 0; x4 < 4; ++x4)
                        st_smem_v4(p_at + (((k * 4 + x4) ^ (i & 7)) << 4),
                                   make_uint4(v[k][4 * x4], v[k][4 * x4 + 1], v[k][4 * x4 + 2], v[k][4 * x4 + 3]));
                fence_async_smem();
                tc_fence_before();
                tell(weighed_at);
            }
            // (a break leaves the loop with both warps, and so does this)
            ok = ok && all(mbar_wait(bar(sm.added), (n - 1) & 1, gave_up));
            tc_fence_after();
            const float part_lse = a.part ? a.part_lse[at.n] : 0.0f;      // (lse may be the same)
            sm.sum[half][i] = l;
            if (!(ok = meet(ok))) break;
            l += sm.sum[half ^ 1][i];
            meet(true);
            if (t0 == 0 && t1 == w.tiles) {      // the heads' whole sums
                float weight = 0.0f, scale = 1.0f;
                const uint8_t *part = nullptr;
                if (a.part) {
                    scale = add_part(m, l, part_lse, &weight);
                    if (weight != 0.0f) part = a.part + at.r * a.part_rs + at.h * a.part_hs + half * 512;
                }
                const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
                if (on && half == 0 && a.lse) a.lse[at.n] = log2_sum(m, l) * kLn2;
                scale *= inv;
                weight *= inv;
                uint8_t *out = a.out + at.r * a.out_rs + at.h * a.out_hs + half * 512;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t o[32];
                    tmem_ld_32(lanes + T_O + c, o);
                    tmem_wait_ld();
                    if (!on) continue;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float x[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[8 * j + k]);
                        uint4 p = make_uint4(0, 0, 0, 0);
                        if (part) p = ld_dev_v4(part + c * 2 + j * 16);
                        st_v4(out + c * 2 + j * 16, weighted8<DT>(x, scale, p, weight, part != nullptr));
                    }
                }
            } else {
                const int64_t place = ((int64_t)pair * 2 + (t0 == 0)) * PAIR_HEADS + rank * CTA_HEADS + i;
                if (half == 0) w.ml[place] = make_float2(m, l);
                float *o_at = w.o + place * kLatent + half * 256;
#pragma unroll 1
                for (int c = 0; c < 256; c += 32) {
                    uint32_t o[32];
                    tmem_ld_32(lanes + T_O + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        *reinterpret_cast<uint4 *>(o_at + c + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
                }
            }
            tc_fence_before();
        }
    }
    __syncwarp();
    if (sm.gave_up) {      // let copies in flight come in (16 KB each, microseconds)
        uint64_t t0, t;
        asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
        do {
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
        } while (t - t0 < 1000000ull);
    }
    tc_fence_before();
    __syncthreads();
    pair_sync();      // no CTA leaves before the other has done with it
    if (tid == 0 && sm.gave_up && a.status)
        for (int r = 0; r < a.R; ++r) record_status(a.status, r, kStatusAttendTimeout);
    if (warp == MMA_WARP) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ---- join ------------------------------------------------------------------------------

constexpr int JOIN_NT = 128;

// A warp a head: its parts from the pairs that have some of its tiles.
template <int DT>
__global__ void __launch_bounds__(JOIN_NT) join_kernel(const __grid_constant__ PrefixLaunch a, const __grid_constant__ PrefixParts w)
{
    const int lane = threadIdx.x & 31;
    const int64_t head = (int64_t)blockIdx.x * (JOIN_NT / 32) + (threadIdx.x >> 5);
    after_launch_before();
    if (head >= (int64_t)a.R * a.H) return;
    const HeadPlace at(a, head);
    const int group = (int)(head / PAIR_HEADS), i = (int)(head % PAIR_HEADS);
    const int64_t begin = (int64_t)group * w.tiles;
    int p0 = 0, p1 = -1;
    if (w.units > 0) {
        p0 = pair_of(w, begin);
        p1 = pair_of(w, begin + w.tiles - 1);
        if (p0 == p1) return;      // (that pair has written it)
    }
    auto place = [&](int p) { return ((int64_t)p * 2 + (first_unit(w, p) <= begin)) * PAIR_HEADS + i; };
    float m = -INFINITY;
    for (int p = p0; p <= p1; ++p) m = fmaxf(m, w.ml[place(p)].x);
    const float base = m == -INFINITY ? 0.0f : m;
    float l = 0.0f, o[2][8] = {};
    for (int p = p0; p <= p1; ++p) {
        const float2 ml = w.ml[place(p)];
        const float f = ex2(ml.x - base);
        l = fmaf(f, ml.y, l);
        const float *src = w.o + place(p) * kLatent + lane * 8;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const float4 x = *reinterpret_cast<const float4 *>(src + k * 256 + j);
                o[k][j] = fmaf(f, x.x, o[k][j]);
                o[k][j + 1] = fmaf(f, x.y, o[k][j + 1]);
                o[k][j + 2] = fmaf(f, x.z, o[k][j + 2]);
                o[k][j + 3] = fmaf(f, x.w, o[k][j + 3]);
            }
    }
    float weight = 0.0f, scale = 1.0f;
    uint4 part[2] = {};
    if (a.part) {
        const uint8_t *src = a.part + at.r * a.part_rs + at.h * a.part_hs + lane * 16;
        part[0] = ld_dev_v4(src);
        part[1] = ld_dev_v4(src + 512);
        scale = add_part(m, l, a.part_lse[at.n], &weight);
    }
    const float inv = l == 0.0f ? 0.0f : __fdividef(1.0f, l);
    uint8_t *out = a.out + at.r * a.out_rs + at.h * a.out_hs + lane * 16;
    __syncwarp();      // (part may be out, part_lse lse)
#pragma unroll
    for (int k = 0; k < 2; ++k)
        st_v4(out + k * 512, weighted8<DT>(o[k], scale * inv, part[k], weight * inv, weight != 0.0f));
    if (lane == 0 && a.lse) a.lse[at.n] = log2_sum(m, l) * kLn2;
}

// ---- host ------------------------------------------------------------------------------

PrefixParts lay_out(int32_t R, int32_t H, int32_t len, uint8_t *ws, int64_t *bytes)
{
    PrefixParts w = {};
    w.tiles = (len + KEYS - 1) / KEYS;
    w.groups = (int)(((int64_t)R * H + PAIR_HEADS - 1) / PAIR_HEADS);
    w.units = (int64_t)w.tiles * w.groups;
    w.pairs = (int)(w.units < MAX_PAIRS ? w.units : MAX_PAIRS);
    int64_t n = 16;      // never empty
    w.o = reinterpret_cast<float *>(ws + n);
    n += (int64_t)w.pairs * 2 * PAIR_HEADS * kLatent * 4;
    w.ml = reinterpret_cast<float2 *>(ws + n);
    n += (int64_t)w.pairs * 2 * PAIR_HEADS * 8;
    w.there = reinterpret_cast<uint32_t *>(ws + n);
    n += (int64_t)w.tiles * 16;
    n = (n + 127) / 128 * 128;
    w.image = ws + n;
    n += (int64_t)w.tiles * TILE_BYTES;
    *bytes = n;
    return w;
}

// Sets the kernels' attributes on the current device, once.
cudaError_t prepare_device()
{
    constexpr int kDevices = 64;
    static std::atomic<bool> known[kDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= kDevices) return cudaErrorInvalidDevice;
    if (!known[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(prefix_kernel<kBf16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PX_SMEM);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(prefix_kernel<kF16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PX_SMEM);
        if (e != cudaSuccess) return e;
        known[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

template <int DT>
cudaError_t launch(const PrefixLaunch &a, const PrefixParts &w, cudaStream_t s)
{
    if (w.units > 0) {
        auto expand = a.row_bytes == kRow4 ? expand_kernel<DT, kRow4> : a.row_bytes == kRow8 ? expand_kernel<DT, kRow8> : expand_kernel<DT, kRow16>;
        cudaError_t e = launch_behind(expand, dim3(w.tiles * (KEYS / EX_KEYS)), EX_NT, 0, 1, s, a, w);
        if (e != cudaSuccess) return e;
        e = launch_behind(prefix_kernel<DT>, dim3(w.pairs * 2), PX_NT, PX_SMEM, 2, s, a, w);
        if (e != cudaSuccess) return e;
        bool split = false;
        for (int p = 1; p < w.pairs; ++p) split = split || first_unit(w, p) % w.tiles != 0;
        if (!split) return e;
    }
    return launch_behind(join_kernel<DT>, dim3((unsigned)(((int64_t)a.R * a.H + JOIN_NT / 32 - 1) / (JOIN_NT / 32))), JOIN_NT, 0, 1, s, a, w);
}

}  // namespace

void attend_prefix_workspace_bytes(int32_t R, int32_t H, int32_t len, int64_t *bytes) { lay_out(R, H, len, nullptr, bytes); }

cudaError_t launch_attend_prefix(const PrefixLaunch &a, cudaStream_t s)
{
    const cudaError_t e = prepare_device();
    if (e != cudaSuccess) return e;
    int64_t bytes;
    const PrefixParts w = lay_out(a.R, a.H, a.len, a.workspace, &bytes);
    return a.dtype == kBf16 ? launch<kBf16>(a, w, s) : launch<kF16>(a, w, s);
}

}  // namespace hs
